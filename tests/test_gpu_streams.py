"""GPU: calls on another stream than the one their tensors belong to. A side stream is kept busy, the call is
enqueued behind that, and what the caller's stream allocates and fills meanwhile must be other memory than the
call still uses: the call's results are right, and the fills stay as they are."""
import pytest
import torch

from speculative_decoding_verification_43_gb300 import api, workloads as W

from attend_ref import Batch
import test_gpu_append as A

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def busy_stream():
    """A stream with some milliseconds of work ahead."""
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    return st


def fills(*tensors):
    """Tensors of the given ones' sizes (several of each), allocated and filled on the current stream."""
    return [torch.full((t.numel() * t.element_size(),), 0xA5, dtype=torch.uint8, device="cuda")
            for t in tensors for _ in range(3)]


def untouched(tensors):
    return all(bool((t == 0xA5).all()) for t in tensors)


def batch(kv=(900, 1300, 40)):
    return Batch([3, 5, 1], list(kv), 8, 2, 128, BF, 16, shared=32, seed=1).place()


def attend_once(b, **kw):
    return api.attend(b.qd, b.k_cache, b.v_cache, b.row_off, b.kv_len, b.table, shared_len=b.shared,
                      shared_table=b.shared_table, **kw)


def settled(b):
    """The call's results on the current stream, and tensors of its outputs' and workspace's sizes."""
    a = b.attention()
    o = a.run()
    want = o.out.clone(), o.lse.clone()
    like = [torch.empty_like(t) for t in (a.workspace, o.out, o.lse, o.req_status)]
    torch.cuda.synchronize()
    return want, like


def test_attend_on_a_busy_stream():
    b = batch()
    want, like = settled(b)
    st = busy_stream()
    o = attend_once(b, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert torch.equal(o.out, want[0]) and torch.equal(o.lse, want[1])
    assert untouched(f)


def test_attend_on_a_busy_stream_result_dropped():
    b = batch()
    _, like = settled(b)
    st = busy_stream()
    attend_once(b, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def test_attend_outputs_still_read_when_dropped():
    """The caller's stream is behind with reading the outputs while their own stream allocates again."""
    b = batch()
    want, like = settled(b)
    st, here = torch.cuda.Stream(), torch.cuda.current_stream()
    st.wait_stream(here)
    o = attend_once(b, stream=st)
    here.wait_stream(st)
    torch.cuda._sleep(20_000_000)
    x, y = o.out.clone(), o.lse.clone()
    del o
    with torch.cuda.stream(st):
        f = fills(*like)
    torch.cuda.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(y, want[1]) and untouched(f)


def test_prepared_attention_dropped_while_it_runs():
    b = batch()
    _, like = settled(b)
    a = b.attention()
    st = busy_stream()
    a.run(st)
    del a
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def test_prepared_attention_with_its_stream_made_current():
    b = batch()
    _, like = settled(b)
    a = b.attention()
    with torch.cuda.stream(busy_stream()):
        a.run()
    del a
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def test_prepared_attention_bound_anew_while_it_runs():
    """A larger call's workspace takes the place of the one still in use."""
    b, big = batch(), Batch([3, 5, 1], [900, 1300, 40], 8, 2, 128, BF, 16, shared=32, seed=2).place()
    want, like = settled(b)
    a = b.attention()
    st = busy_stream()
    out = a.run(st).out
    a.workspace, a.ws_bytes, old = None, 0, a.workspace.numel()
    a.bind(big.qd, big.k_cache, big.v_cache, big.row_off, big.kv_len, big.table, shared_table=big.shared_table,
           out=torch.empty_like(out))
    assert a.workspace.numel() >= old
    f = fills(*like)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and untouched(f)


def test_kv_append_on_a_busy_stream():
    a, _ = A.make([3, 2], [60, 70], 4, 2, 64, BF, 16, 64)
    o = api.kv_append(**a)
    want, k = o.q.clone(), a["k_cache"].clone()
    like = [torch.empty_like(o.q), torch.empty_like(o.req_status)]
    torch.cuda.synchronize()
    st = busy_stream()
    o = api.kv_append(**a, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert torch.equal(o.q, want) and torch.equal(a["k_cache"], k) and untouched(f)
    st = busy_stream()
    api.kv_append(**a, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def test_prepared_append_dropped_while_it_runs():
    a, _ = A.make([3, 2], [60, 70], 4, 2, 64, BF, 16, 64)
    c = api.KvAppender(2, 5, 4, 2, 64, BF).bind(**a)
    like = [torch.empty_like(c.out.q), torch.empty_like(c.out.req_status)]
    st = busy_stream()
    c.run(st)
    del c
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def verifier_round():
    rd = W.make_round(W.Workload("busy", B=12, V=20000, dtype=BF, temperature=0.7, logits="zipf", sigma=1.0,
                                 draft_sigma=0.8, K="uniform:0:7"), seed=1, rnd=0, device="cuda")
    return rd, (rd.target, rd.draft, rd.row_off, rd.draft_tokens, rd.uniforms, rd.temperature)


@pytest.mark.parametrize("keep", [True, False], ids=["kept", "dropped"])
def test_verify_on_a_busy_stream(keep):
    _, args = verifier_round()
    v = api.Verifier(args[2].numel() - 1, args[0].shape[1], args[0].shape[0], BF).bind(*args)
    o = v.run()
    want = [o.accept_len.clone(), o.out_tokens.clone(), o.alpha_rows.clone()]
    like = [torch.empty_like(t) for t in (v.workspace, o.out_tokens, o.alpha_rows)]
    torch.cuda.synchronize()
    st = busy_stream()
    o = api.verify(*args, stream=st)
    if not keep:
        del o
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)
    if keep:
        assert all(torch.equal(x, y) for x, y in zip((o.accept_len, o.out_tokens, o.alpha_rows), want))


def test_compact_and_the_gamma_choice_on_a_busy_stream():
    rd, args = verifier_round()
    o = api.verify(*args)
    ci = W.make_compaction_inputs(rd, 64, 16)
    ins = (rd.row_off, o.accept_len, o.n_emitted, o.out_tokens, o.req_status, ci["prefix_len"], ci["cand_kv_rows"],
           ci["block_table"], ci["page_size"])
    want, (g, a) = api.compact(*ins), api.choose_gamma(o.alpha_sum, o.alpha_count, 0.5, 0.05)
    like = [torch.empty_like(t) for t in vars(want).values()]
    torch.cuda.synchronize()
    st = busy_stream()
    c = api.compact(*ins, stream=st)
    g2, a2 = api.choose_gamma(o.alpha_sum, o.alpha_count, 0.5, 0.05, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    n = int(want.out_off[-1])
    assert torch.equal(c.out_off, want.out_off) and torch.equal(c.packed_tokens[:n], want.packed_tokens[:n])
    assert torch.equal(g2, g) and torch.equal(a2, a) and untouched(f)


def test_a_round_dropped_while_it_runs():
    rd, args = verifier_round()
    ci = W.make_compaction_inputs(rd, 64, 16)
    v = api.Verifier(rd.B, args[0].shape[1], rd.T, BF).bind(*args)
    c = api.Compactor(rd.B, rd.T).bind(rd.row_off, v.out.accept_len, v.out.n_emitted, v.out.out_tokens, v.out.req_status,
                                       ci["prefix_len"], ci["cand_kv_rows"], ci["block_table"], ci["page_size"])
    like = [torch.empty_like(t) for t in (v.workspace, v.out.out_tokens, c.out.packed_tokens, c.out.out_off)]
    st = busy_stream()
    api.run_round(v, c, 0.5, 0.05, stream=st)
    del v, c
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)
