"""GPU tests of calls on a given stream while the current stream is busy: blocks that were
freed on the current stream are still written by a kernel queued there, and the caller
goes on with outputs on the current stream and frees them. Neither may reach what a call
allocates (see test_stream_alloc_host.py for which allocations that is)."""
import pytest
import torch

import test_gpu_norm_rope
import test_gpu_quant_cache
import test_gpu_tree_attn

pytestmark = pytest.mark.gpu
BUSY = 300_000_000   # clock cycles: about 150 ms, far longer than the calls take


@pytest.fixture(scope="module")
def api():
    from learned_token_pruning_gemm_b200 import api, build
    build.build()
    api.device_status(reset=True)
    return api


def _norm(api):
    q, k, wq, wk, pos, dq, dk = test_gpu_norm_rope._inputs(5, 300, 4, 2, 128, torch.bfloat16, False)
    need = api.qk_norm_rope_bwd_workspace_size(300, 4, 2, 128)
    return (lambda **kw: api.qk_norm_rope(q, k, wq, wk, pos, **kw) + api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, **kw),
            [q.nbytes, k.nbytes, q.nbytes, k.nbytes, wq.nbytes, wk.nbytes, need])


def _read(api):
    c = test_gpu_quant_cache._empty(2, 500, 4, 128, torch.int8)
    ln, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([400, 333], [0, 400, 733]))
    return (lambda **kw: api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, cu, 733, **kw),
            [733 * 4 * 128 * 2, 733 * 4 * 128 * 2, 733 * 4])


def _tree(fmt, T):
    def make(api):
        st = test_gpu_tree_attn.make(6, 2, T, 700, [700, 311], 8, 4, 128, fmt, garbage=False)
        need = api.tree_attention_workspace_size(2, T, 8, 4, 128, 700)
        return (lambda **kw: (test_gpu_tree_attn.run(api, st, max_len=700, **kw),), [st["q"].nbytes, need])
    return make


def _gated(api):
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    K, hq, hkv, dh = 400, 4, 2, 128
    q, k, v, do = (rnd(K, h, dh).to(torch.bfloat16) for h in (hq, hkv, hkv, hq))
    s, gain, tau, lse = rnd(K), rnd(hq).abs(), 0.8 + rnd(hq).abs(), torch.empty(hq, K).cuda()
    cu = torch.tensor([0, 150, 400], dtype=torch.int32).cuda()

    def call(**kw):
        o = api.gated_attention(q, k, v, s, gain, tau, cu, 250, lse=lse, **kw)
        return (o,) + api.gated_attention_bwd(q, k, v, o, do, lse, s, gain, tau, cu, 250, **kw)
    need = api._lib.load().tg_gated_attention_bwd_workspace_size(api.TG_BF16, 2, K, 250, hq, hkv, dh)
    return call, [q.nbytes, q.nbytes, k.nbytes, v.nbytes, s.nbytes, gain.nbytes, tau.nbytes, need]


CASES = {"gated attention": _gated, "norm": _norm, "read": _read, "tree, few rows": _tree(torch.int8, 4), "tree": _tree(torch.bfloat16, 64)}


@pytest.mark.parametrize("name", sorted(CASES))
def test_busy_current_stream(api, name):
    call, sizes = CASES[name](api)
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=s)   # loading kernels and asking the device for memory would wait for it later
    # blocks of the sizes that the call allocates: freed, but written once the stream gets to it
    blocks = [torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for b in blocks:
        b.fill_(254)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for b in blocks:
        b.fill_(255)
    places = {b.untyped_storage().data_ptr() for b in blocks}
    blocks.clear()
    del b
    got = call(stream=s)
    late = torch.cuda.Event()
    late.record()
    s.synchronize()
    busy = not late.query()   # the call was over before the fills ran: they come last
    torch.cuda.synchronize()
    assert busy, "the current stream was meant to be busy all the while"
    assert not places & {t.untyped_storage().data_ptr() for t in got}
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # outputs freed while the current stream has yet to read them stay as they are until then
    torch.cuda._sleep(BUSY)
    kept = [t.clone() for t in got]
    del got
    more = [call(stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    for got in more:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert api.device_status(reset=True) == 0


@pytest.mark.parametrize("name", sorted(CASES))
def test_captured_on_a_forked_stream(api, name):
    # inside a capture, on a second stream that joins it: what the call allocates is the graph's, its
    # outputs are used on the first stream and freed, and the call comes again
    call, _ = CASES[name](api)
    want = [t.clone() for t in call()]
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    call(stream=second)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=first):
        kept = []
        for _ in range(3):
            second.wait_stream(first)
            got = call(stream=second)
            first.wait_stream(second)
            kept.append([t.clone() for t in got])
            del got
    for _ in range(3):
        for ts in kept:
            for t in ts:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for ts in kept for a, b in zip(ts, want))
    assert api.device_status(reset=True) == 0
