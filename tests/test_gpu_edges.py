"""Edge cases of the entry points on the GPU: calls with no keys at all."""
import pytest
import torch

from scaled_dot_product_prefill_b200 import api, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_with_no_keys_gives_zeros_and_minus_infinity_lse(dtype):
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = inputs.normal((2, 4, 70, 64), seed=1, dtype=dtype).cuda()
    k = torch.empty((2, 2, 0, 64), dtype=tdt, device="cuda")
    v = torch.empty_like(k)
    fn = api.attn_prefill_lse if dtype == "bf16" else api.attn_prefill_f32_lse
    out, lse = fn(q, k, v, causal=False)
    torch.cuda.synchronize()
    assert (out == 0).all()
    assert torch.isneginf(lse).all()


def test_paged_prefill_and_decode_with_empty_caches():
    p = inputs.paged_inputs(3, 8, 2, 128, 16, seed=3, seq_lens=[0, 0, 0], max_pages=2)
    # the pools need at least one page to have an address; nothing is read from them
    kp = torch.zeros((1, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = inputs.normal((3, 8, 5, 128), seed=4).cuda()
    out, lse = api.attn_prefill_paged(q, kp, kp, table, lens, max_seq_len=0, want_lse=True)
    qd = p.q.cuda()
    dec = api.attn_decode_paged(qd, kp, kp, table, lens, max_seq_len=0)
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert (dec == 0).all()


def test_append_of_nothing_is_a_no_op():
    kp = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    before = kp.clone()
    k_new = torch.empty((2, 2, 0, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    api.attn_kv_append(k_new, k_new, kp, kp, table, lens)
    torch.cuda.synchronize()
    assert torch.equal(kp, before)


def test_calls_on_another_stream_are_not_overwritten_by_work_queued_on_this_one():
    """The current stream still has to fill blocks that were released on the host: no result or scratch of a
    call on another stream may lie in them."""
    inp = inputs.prefill_inputs(1, 8, 2, 500, 500, 64, seed=4)
    q, k, v = inp.q.cuda(), inp.k.cuda(), inp.v.cuda()
    host = [x.pin_memory() for x in (inp.q, inp.k, inp.v)]
    p = inputs.paged_inputs(3, 8, 2, 64, 16, seed=6, seq_lens=[1500, 900, 77])
    dq, kp, vp, pt, sl = (x.cuda() for x in (p.q, p.k_pool, p.v_pool, p.page_table, p.seq_lens))
    new = [x.pin_memory() for x in (p.q, inputs.normal((3, 2, 1, 64), 8), inputs.normal((3, 2, 1, 64), 9))]

    def calls(**kw):
        return [api.attn_prefill(q, k, v, causal=True, **kw), *api.attn_prefill_lse(q, k, v, **kw),
                api.attn_prefill_f32(q.float(), k.float(), v.float(), **kw),
                api.attn_decode_paged(dq, kp, vp, pt, sl, max_seq_len=1500, **kw),
                api.attn_prefill_host(*host, causal=True, **kw),
                api.attn_decode_step_host(*new, kp, vp, pt, sl, max_seq_len=1500, **kw)]

    calls()                                    # (the step appends its token: the same one below)
    want = calls()
    need = api.attn_decode_paged_workspace_size(3, 8, 64, 1500, 16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(200_000_000)             # some 100 ms
    for _ in range(3):
        for size in (2 * q.numel(), 4 * q.numel(), 2 * k.numel(), 8 * 500 * 4, 2 * dq.numel(), 2 * new[1].numel(), need):
            torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    with torch.cuda.stream(s):
        f32 = [x.float() for x in (q, k, v)]
    got = [api.attn_prefill(q, k, v, causal=True, stream=s), *api.attn_prefill_lse(q, k, v, stream=s),
           api.attn_prefill_f32(*f32, stream=s), api.attn_decode_paged(dq, kp, vp, pt, sl, max_seq_len=1500, stream=s),
           api.attn_prefill_host(*host, causal=True, stream=s),
           api.attn_decode_step_host(*new, kp, vp, pt, sl, max_seq_len=1500, stream=s)]
    torch.cuda.synchronize()
    assert api.attn_device_status(clear=True) == 0
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i
