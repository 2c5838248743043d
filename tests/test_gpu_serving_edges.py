"""Serving operators at the edges of their contracts, against the plain 64-bit forms (tests/serving_helpers.py):
query rows that are not finite, offsets that decrease next to sound ones, float32 sums over very long rows.
Tolerances: tests/test_gpu_serving.py, unless a test derives its own."""
import numpy as np
import pytest
import torch

import serving_helpers as R
from gpu_helpers import BF, lib
from test_gpu_serving import F32, U32, UBF, Prompt, check_out, check_weight, host, i32, score_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("n_q,n_kv,row", [(400, 400, 264), (400, 400, 265), (400, 400, 266), (400, 400, 3), (450, 480, 384),
                                          (5, 2500, 0), (5, 2500, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prompt_nonfinite_query_row(cuda, kernel, dtype, d, n_q, n_kv, row, value):
    """One query row of one head is not finite: its output and the weights of every key that it sees are NaN,
    wherever the row lies in a tile; all else is as without it."""
    p = Prompt(lib(), dtype, d, 2, 2, [n_q], [n_kv], seed=row + d, kernel=kernel)
    q = host(p.q)
    q[row, 0] = 0
    p.q[row, 0, :3] = value
    p.run()
    k, v = host(p.k), host(p.v)
    ref, w = R.prompt_attention(q, k, v, p.cu_q, p.cu_kv, p.n_w)
    spread, _ = R.prompt_attention(q, k, np.abs(v), p.cu_q, p.cu_kv, p.n_w)
    e, seen = score_step(q, k, n_kv), row + n_kv - n_q + 1
    o, got = host(p.o), host(p.w)
    assert np.isnan(o[row, 0]).all() and np.isnan(got[0, 0, :seen]).all()
    o[row, 0], ref[row, 0] = 0, 0
    check_out(o, ref, spread, e, dtype, UBF if dtype == BF and kernel == 0 else 0.0)
    check_weight(got[0, 0, seen:], host(p.w0)[0, 0, seen:], w[0, 0, seen:], e)
    check_weight(got[0, 1], host(p.w0)[0, 1], w[0, 1], e)


OUTSIDE = 10 ** 6   # an offset that leaves the block
MANY = [5 * b for b in range(41)]
MANY[20] = OUTSIDE


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
@pytest.mark.parametrize("cu_q,cu_kv", [
    ([30, 20, 50], [30, 20, 50]), ([0, 40, 100, 60], [0, 40, 100, 60]), ([0, 5, OUTSIDE, 5, 100], [0, 5, OUTSIDE, 5, 100]),
    ([7, 7, 2, 9], [0, 3000, 3000, 7000]), ([0, 3, 6, 4], [0, 4000, 8000, 8000]),
    ([0, 3, 9], [4000, 3000, 9000]), ([0, 5, -1, 5, 8], [0, 2000, 4000, 4000, 8000]), (MANY, MANY)])
def test_prompt_sound_sequences_next_to_bad_offsets(cuda, dtype, H, Hk, cu_q, cu_kv):
    """Offsets that decrease or leave their block make their own sequence empty; the others are whole, with
    grouped heads (whose weights a kernel of their own adds up) and with keys split over CTAs too."""
    S, B, d = lib(), len(cu_q) - 1, 64
    top = lambda cu: max(c for c in cu if c != OUTSIDE)
    q_rows, kv_rows = top(cu_q), top(cu_kv)
    p = Prompt(S, dtype, d, H, Hk, [q_rows] + [0] * (B - 1), [kv_rows] + [0] * (B - 1), seed=B + H)
    cq, ck = i32(cu_q), i32(cu_kv)
    p.args.cu_q, p.args.cu_kv = cq.data_ptr(), ck.data_ptr()
    p.run()
    assert int(p.status.item()) == S.E_INDEX
    rows = lambda cu, n, b: (cu[b], cu[b + 1]) if 0 <= cu[b] <= cu[b + 1] <= n else (0, 0)
    q, k, v, o = host(p.q), host(p.k), host(p.v), host(p.o)
    rest = np.ones(q_rows, bool)
    for b in range(B):
        q0, q1 = rows(cu_q, q_rows, b)
        k0, k1 = rows(cu_kv, kv_rows, b)
        one = lambda v: R.prompt_attention(q[q0:q1], k[k0:k1], v, [0, q1 - q0], [0, k1 - k0], p.n_w)
        (ref, w), (spread, _) = one(v[k0:k1]), one(np.abs(v[k0:k1]))
        e = score_step(q[q0:q1], k[k0:k1], k1 - k0)
        check_out(o[q0:q1], ref, spread, e, dtype, UBF if dtype == BF else 0.0, f"sequence {b}")
        check_weight(host(p.w)[b], host(p.w0)[b], w[0], e, f"sequence {b}")
        rest[q0:q1] = False
    assert (o[rest] == 7.0).all(), "rows outside every sequence were written"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [1, 40])
def test_attention_float32_sums_do_not_drift(cuda, d, B):
    """Float32 queries over 16,000 rows, values of one sign: sums that cut their last bits off fall short by a part
    that grows with the rows (kept in the tensor cores over a whole sequence, 1.6e-6; over an eighth of it, 5.4e-7).
    One sequence, and so many that one CTA sums most of a sequence (all have the same rows and queries of their
    own).  The scores are below 4 and each output is a mean of about n values with independent errors: rounded
    to nearest they are 2**-22 or so each (scores, exponentials), and their mean over all outputs is far below
    that: 2**-21 is left for it, and 2**-19 for a single output."""
    S, Hk, n = lib(), 8, 16000
    r = np.random.default_rng(d)
    codes = [r.integers(-7, 8, (n, d)), r.integers(1, 8, (n, d))]
    scales = [R.to_bf16(np.exp(r.normal(0, 0.3, (n, d // 32)))) for _ in range(2)]
    dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda().expand(B, Hk, *a.shape).contiguous()
    t = [dev(R.pack4(codes[0], 8), torch.uint8), dev(scales[0], BF), dev(R.pack4(codes[1], 4), torch.uint8), dev(scales[1], BF)]
    w = torch.zeros((B, Hk, n), device="cuda")
    c = S.make_kv4_cache(*t, w)
    k, v = (a * np.repeat(s.astype(np.float64), 32, -1) for a, s in zip(codes, scales))
    q = torch.randn((B, Hk, d), generator=torch.Generator(device="cuda").manual_seed(d), device="cuda") * 0.08
    o, status = torch.empty_like(q), i32([0])
    a = S.make_kv4_attn_args(c, q, o, i32([n] * B), n, dev_status=status)
    nb = S.kv4_attention_workspace_size(a)
    S.kv4_attention(a, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    qh = host(q).reshape(-1, d)
    x = qh @ k.T / np.sqrt(d)
    assert np.abs(x).max() < 4
    p = R.softmax_rows(x)
    ref = p @ v
    rel = host(o).reshape(-1, d) / ref - 1
    assert int(status.item()) == 0
    assert abs(rel.mean()) <= 2.0 ** -21 and np.abs(rel).max() <= 2.0 ** -19
    assert abs(host(w).sum() / p.sum() - 1) <= 2.0 ** -21


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_prompt_over_rows_and_resume_of_other_counts_are_reported(cuda, dtype, H, Hk):
    """A prompt's weights belong to an empty sequence's first rows, a resumed one's to as many rows as the cache
    holds: elsewhere they would go to other tokens' rows.  Such sequences are reported and add none; those next
    to them, one without new rows among them, are served."""
    from cascade_token_head_b200.kv4 import KV4State
    S, d, B = lib(), 64, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda r, h: torch.randn((r, h, d), generator=g, device="cuda").to(dtype)
    st = KV4State(B, H, Hk, d, 64)
    st.prompt(rnd(30, H), rnd(30, Hk), rnd(30, Hk), i32([0, 20, 30, 30]))
    assert int(st.status.item()) == 0 and st.len.tolist() == [20, 10, 0]
    w = st.weight.clone()
    q, k, v = rnd(12, H), rnd(12, Hk), rnd(12, Hk)
    st.prompt(q, k, v, i32([0, 0, 5, 12]))                    # sequence 1 held rows, 2 held none
    assert int(st.status.item()) == S.E_INDEX and st.len.tolist() == [20, 15, 7]
    assert torch.equal(st.weight[:2], w[:2])
    _, add = R.prompt_attention(host(q)[5:], host(k)[5:], host(v)[5:], [0, 7], [0, 7], 64)
    check_weight(host(st.weight)[2], 0.0, add[0], score_step(host(q), host(k), 7))
    st.status.zero_()
    w = st.weight.clone()
    st.resume(rnd(3, H), rnd(3, Hk), rnd(3, Hk), i32([0, 1, 2, 3]), i32([0, 21, 37, 44]), 44)   # sequence 2: 7 for 8
    assert int(st.status.item()) == S.E_INDEX and st.len.tolist() == [21, 16, 8]
    assert torch.equal(st.weight[2], w[2]) and (st.weight[:2] != w[:2]).any(2).all()
    st.status.zero_()
    st.resume(rnd(3, H), rnd(3, Hk), rnd(3, Hk), i32([0, 1, 2, 3]), i32([0, 22, 39, 48]), 48)
    assert int(st.status.item()) == 0
    st = KV4State(B, H, Hk, d, 16)                            # rows that do not fit are dropped, the others' weights are kept
    q, k, v = rnd(25, H), rnd(25, Hk), rnd(25, Hk)
    st.prompt(q, k, v, i32([0, 20, 25, 25]))
    assert int(st.status.item()) == S.E_INDEX and st.len.tolist() == [16, 5, 0]
    _, add = R.prompt_attention(host(q), host(k), host(v), [0, 20, 25], [0, 20, 25], 16)
    check_weight(host(st.weight)[:2], 0.0, add, score_step(host(q), host(k), 20))


@pytest.mark.parametrize("dtype,kernel", [(BF, 0), (BF, 1), (F32, 0), (F32, 1)])
@pytest.mark.parametrize("H,Hk", [(2, 2), (6, 2)])
def test_prompt_weights_of_counted_rows(cuda, dtype, kernel, H, Hk):
    S = lib()
    lens, kv = [5, 0, 140, 3], [40, 9, 140, 3000]
    p = Prompt(S, dtype, 64, H, Hk, lens, kv, seed=3, kernel=kernel)
    held = i32([40, 1, 139, 3000])
    p.args = S.make_prompt_args(p.q, p.k, p.v, p.o, i32(p.cu_q), i32(p.cu_kv), weight=p.w, dev_status=p.status, kernel=kernel, weight_len=held)
    p.run()
    assert int(p.status.item()) == S.E_INDEX and torch.equal(p.w[2], p.w0[2])
    q, k, v = host(p.q), host(p.k), host(p.v)
    _, w = R.prompt_attention(q, k, v, p.cu_q, p.cu_kv, p.n_w)
    w[2] = 0
    check_weight(host(p.w), host(p.w0), w, score_step(q, k, 3000))
    held.copy_(i32([40, 1, 140, 3000]))
    p.w.copy_(p.w0)
    p.status.zero_()
    p.run().check(UBF if dtype == BF and kernel == 0 else 0.0)
