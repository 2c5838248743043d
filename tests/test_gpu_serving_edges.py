"""Serving operators at the edges of their contracts, against the plain 64-bit forms (tests/serving_helpers.py):
query rows that are not finite, offsets that decrease next to sound ones, float32 sums over very long rows.
Tolerances: tests/test_gpu_serving.py, unless a test derives its own."""
import numpy as np
import pytest
import torch

import serving_helpers as R
from gpu_helpers import BF, lib
from test_gpu_serving import Cache, F32, U32, UBF, Prompt, check_out, check_weight, host, i32, score_step

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


def norm_error(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


# A float32 call with scores below about 4 errs by independent roundings: of a score (2**-24 of it from each of the
# query's terms, the product and its scaling, 2**-22 in all), its exponential (2**-22), sums of partial sums that
# are much smaller than 2**-24 times their number, the quotient.  Their root mean square over all outputs is below
# 2**-21; 2**-20 is left.  An operand term that gets lost costs 2**-16 or more (the bfloat16 terms: 2**-8, 2**-16
# of a value; the query's fp16 terms: 2**-11).  The CUDA-core prompt kernel adds a row's n products one by one: sums
# of terms of both signs grow like the root of their number, so step k rounds by at most 2**-24 sqrt(k / n) of the
# result, and the root of the sum of their squares is 2**-24 sqrt(n / 2) at most.
FLOAT32_RMS = 2.0 ** -20


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("lens,kv", [([1500, 700], [1500, 700]), ([40], [6000]), ([300], [2300])])
def test_prompt_float32_is_float32(cuda, d, kernel, lens, kv):
    p = Prompt(lib(), F32, d, 4, 2, lens, kv, seed=d, kernel=kernel)
    p.qb *= 0.15
    p.run()
    ref, w = R.prompt_attention(host(p.q), host(p.k), host(p.v), p.cu_q, p.cu_kv, p.n_w)
    assert norm_error(host(p.o), ref) <= FLOAT32_RMS + (U32 * (max(kv) / 2) ** 0.5 if kernel else 0.0)
    assert norm_error(host(p.w), host(p.w0) + w) <= FLOAT32_RMS


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,n", [(1, 2, 20000), (3, 32, 5000), (1, 4, 300)])
def test_attention_float32_is_float32(cuda, d, B, H, n):
    S, Hk = lib(), 2
    r = np.random.default_rng(n)
    code = lambda: r.integers(-7, 8, (Hk, n, d))
    scale = lambda: R.to_bf16(np.exp(r.normal(0, 0.3, (Hk, n, d // 32))))
    kc, vc, ks, vs = code(), code(), scale(), scale()
    dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda().expand(B, *a.shape).contiguous()
    w = torch.zeros((B, Hk, n), device="cuda")
    c = S.make_kv4_cache(dev(R.pack4(kc, 8), torch.uint8), dev(ks, BF), dev(R.pack4(vc, 4), torch.uint8), dev(vs, BF), w)
    k, v = (a * np.repeat(s.astype(np.float64), 32, -1) for a, s in ((kc, ks), (vc, vs)))
    q = torch.randn((B, H, d), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") * 0.15
    o = torch.empty_like(q)
    a = S.make_kv4_attn_args(c, q, o, i32([n] * B), n)
    nb = S.kv4_attention_workspace_size(a)
    S.kv4_attention(a, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    refs = [R.kv4_attention(host(q)[b], k, v, n) for b in range(B)]
    assert norm_error(host(o), np.stack([x for x, _ in refs])) <= FLOAT32_RMS
    assert norm_error(host(w), np.stack([x for _, x in refs])) <= FLOAT32_RMS


# Values at the end of the range that the sums take (|v| < 2**120 / n): the first keys score 0 and all behind
# score just under 2**8 times as much in probability, which the running maximum of the first keys lets pass.
LAG = 7.9 * np.log(2)


@pytest.mark.parametrize("dtype,kernel", [(BF, 0), (BF, 1), (F32, 0), (F32, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n", [(2, 2000), (600, 600)])
def test_prompt_largest_values(cuda, dtype, kernel, d, n_q, n):
    p = Prompt(lib(), dtype, d, 2, 2, [n_q], [n], seed=1, kernel=kernel)
    p.qb.zero_()
    p.kb.zero_()
    p.q[:, :, 0], p.k[128:, :, 0] = 1.0, LAG * d ** 0.5
    p.vb.copy_(0.98 * 2.0 ** 120 / n * (1 - 0.02 * torch.rand(p.vb.shape, device="cuda")))
    p.run().check(UBF if dtype == BF and kernel == 0 else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n", [(1, 2000), (160, 3000)])
def test_attention_largest_values(cuda, dtype, d, B, n):
    S, Hk = lib(), 2
    k, v = np.zeros((n, d), np.int64), np.full((n, d), 7)
    k[:, 0] = 7
    ks, vs = np.ones((n, d // 32)), np.full((n, d // 32), R.to_bf16(0.98 * 2.0 ** 120 / n / 7))
    ks[:300] = 2.0 ** -20
    ks[300:] = R.to_bf16(LAG * d ** 0.5 / 7)
    dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda().expand(B, Hk, *a.shape).contiguous()
    c = S.make_kv4_cache(dev(R.pack4(k, 8), torch.uint8), dev(ks, BF), dev(R.pack4(v, 4), torch.uint8), dev(vs, BF),
                         torch.zeros((B, Hk, n), device="cuda"))
    q = torch.zeros((B, 4, d), device="cuda", dtype=dtype)
    q[:, :, 0] = 1
    o = torch.empty_like(q)
    a = S.make_kv4_attn_args(c, q, o, i32([n] * B), n)
    nb = S.kv4_attention_workspace_size(a)
    S.kv4_attention(a, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    kv = [np.broadcast_to(x * np.repeat(s, 32, -1), (Hk, n, d)) for x, s in ((k, ks), (v, vs))]
    ref, w = R.kv4_attention(host(q)[0], *kv, n)
    e = score_step(host(q)[0], kv[0], n)
    for b in (0, B - 1):
        check_out(host(o)[b], ref, np.abs(ref), e, dtype, UBF if dtype == BF else 2 * U32)
        check_weight(host(c._keep[4])[b], 0.0, w, e)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,H,n,keep", [(1, 2, 5000, 2500), (2, 8, 3001, 1600), (4, 8, 1201, 600), (8, 8, 600, 299), (16, 8, 150, 75),
                                        (12, 12, 1300, 1290)])
def test_evict_every_cluster_size(cuda, in_place, B, H, n, keep):
    """Few heads of many rows to many heads of few: one to eight CTAs a head, of each size."""
    S, d, recent = lib(), 64, keep // 9
    c = Cache(S, B, H, d, n, seed=B)
    c.t["weight"].copy_(torch.round(c.t["weight"] * 16) / 16)      # ties
    before = c.host()
    dst = c if in_place else Cache(S, B, H, d, keep, seed=1)
    ln = [n - 7 * b for b in range(B)]
    held, status = i32(ln), i32([0])
    out = held if in_place else torch.zeros_like(held)
    nb = S.kv4_evict_workspace_size(c.c, n, keep)
    S.kv4_evict(c.c, dst.c, held, out, i32(ln), n, keep, recent, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb, dev_status=status)
    got = dst.host()
    for b in range(B):
        for h in range(0, H, 3):
            src = R.evict_sources(before["weight"][b, h], before["pos"][b, h], ln[b], ln[b], keep, recent)
            for key in got:
                np.testing.assert_array_equal(got[key][b, h, :len(src)], before[key][b, h, src], err_msg=f"{key} {b} {h}")
    assert out.tolist() == [min(x, keep) for x in ln] and int(status.item()) == 0
