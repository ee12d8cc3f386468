"""Workspaces that the products' calls share: a graph has its own, so it may be captured and replayed beside
eager calls and other graphs.  Results are compared bit for bit with those of eager calls."""
import threading
import time

import numpy as np
import pytest
import torch

from fp8_quantized_skinny_qpn_amd import synth
from gpu_util import dev, host, log, need_gpu

pytestmark = pytest.mark.gpu


class Given:
    """Stands before the library and notes the workspace of each call; without `launch` nothing is
    launched, and calls that have a workspace at the same time are counted."""

    def __init__(self, lib, launch=True):
        self.lib, self.launch, self.given, self.inside, self.clashes = lib, launch, [], [], 0

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name not in ("qpn_gemm_nvfp4", "qpn_gemm_prefill_nvfp4", "qpn_lmhead_nvfp4", "qpn_lmhead_verify_nvfp4"):
            return f

        def call(*args):
            ws = args[-3].value                    # .., workspace, its bytes, stream
            self.given.append(ws)
            if self.launch:
                return f(*args)
            self.clashes += ws in self.inside
            self.inside.append(ws)
            time.sleep(0.002)                      # (another thread may run)
            self.inside.remove(ws)
            return 0
        return call


@pytest.fixture(scope="module")
def calls():
    """(qpn, the products whose workspaces hold counters or partial sums, their outputs): split-K, cut tiles, argmax."""
    qpn = need_gpu()
    n, k = 1024, 5120
    pw = qpn.pack_nvfp4(dev(synth.weights(n, k, seed=5)))
    x = dev(synth.activations(64, k, seed=6))
    assert qpn.gemm_plan(qpn.OP_GEMM_NVFP4, 8, n, k).splits > 1
    assert qpn.workspace_bytes(qpn.OP_PREFILL_NVFP4, 64, n, k) > 0
    torch.cuda.synchronize()

    def all_of(stream=None):
        return [qpn.gemm(pw, x[:8], stream=stream), qpn.prefill(pw, x, stream=stream),
                *qpn.lmhead_nvfp4(pw, x[:8], stream=stream)]
    return qpn, all_of, [host(t) for t in all_of()]


def same(got, want):
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert np.array_equal(host(g), w)


def test_graphs_have_workspaces_of_their_own(calls, monkeypatch):
    qpn, all_of, want = calls
    stream, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    same(all_of(stream), want)                     # the stream has its workspace
    watch = Given(qpn.lib)
    monkeypatch.setattr(qpn, "lib", watch)
    held = {b.data_ptr() for b in qpn._workspaces.values()}
    graphs, outs = [], []
    for _ in others:
        g = torch.cuda.CUDAGraph()
        before = len(watch.given)
        with torch.cuda.graph(g, stream=stream):
            outs.append(all_of() + all_of())
        mine = set(watch.given[before:])
        assert not mine & held
        held |= mine
        graphs.append(g)
    for rep in range(4):
        log(f"two graphs and eager calls side by side, {rep}")
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, others):
            with torch.cuda.stream(s):
                g.replay()
        same(all_of(stream), want)
        for out in outs:
            same(out[:4], want)
            same(out[4:], want)


def test_a_stream_whose_first_calls_are_captured(calls):
    # the zero-fill of a capture runs when the graph does: eager calls before that need a workspace of their own
    qpn, all_of, want = calls
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    key = (torch.cuda.current_device(), stream.cuda_stream)
    held = qpn._workspaces.get(key)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        out = all_of()
    assert qpn._workspaces.get(key) is held
    log("eager calls on the stream of a capture")
    same(all_of(stream), want)
    assert int(qpn._workspaces[key].count_nonzero()) == 0
    for _ in range(3):
        g.replay()
        same(out, want)
        same(all_of(stream), want)


def test_threads_do_not_share_the_argmax_keys_at_the_same_time(monkeypatch):
    # the lm_head's second launch reads the rows' keys from the workspace: on one stream, the launches of
    # two threads' calls must not come in turn
    qpn = need_gpu()
    n, k = 512, 1024
    pw = qpn.pack_nvfp4(dev(synth.weights(n, k, seed=7)))
    x, draft = dev(synth.activations(4, k, seed=8)), torch.zeros(3, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    qpn.lmhead_nvfp4(pw, x, stream=stream)
    torch.cuda.synchronize()
    watch = Given(qpn.lib, launch=False)
    monkeypatch.setattr(qpn, "lib", watch)
    failed = []

    def work(f):
        try:
            for _ in range(10):
                f()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(f,)) for f in (
        lambda: qpn.lmhead_nvfp4(pw, x, stream=stream), lambda: qpn.lmhead_verify_nvfp4(pw, x, draft, stream=stream))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed and len(watch.given) == 20 and watch.clashes == 0
