"""Host-side checks of the serving operators (no GPU needed): struct layouts, refusals before any
launch, workspace sizes, and the plain forms the GPU tests compare against."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import serving_helpers as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S():
    from cascade_token_head_b200 import build
    build.build()
    from cascade_token_head_b200 import spatten
    return spatten


def test_struct_layout_matches_header(S, tmp_path):
    structs = {"spatten_prompt_args": S.prompt_args, "spatten_kv4_cache": S.kv4_cache,
               "spatten_kv4_attn_args": S.kv4_attn_args}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "spatten.h"', 'int main(void){']
    for cname, py in structs.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    lines.append("return 0;}")
    (tmp_path / "layout.c").write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {tuple(ln.split()[:2]): int(ln.split()[2]) for ln in out.splitlines()}
    for cname, py in structs.items():
        assert got[(cname, "sizeof")] == C.sizeof(py)
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


def _prompt(S, **over):
    a = S.prompt_args()
    a.B, a.H, a.H_kv, a.d_h, a.total_q, a.total_kv, a.cu_q, a.cu_kv = 2, 8, 2, 64, 100, 120, 1 << 12, 1 << 13
    a.dtype, a.q, a.q_ld_tok, a.k, a.v, a.kv_ld_tok = S.BF16, 1 << 20, 512, 1 << 21, 1 << 22, 128
    a.o, a.o_ld_tok = 1 << 23, 512
    a.weight, a.weight_ld_seq, a.weight_ld_head, a.weight_cap = 1 << 24, 2 * 128, 128, 128
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_prompt_refusals(S):
    call = lambda a, ws=1 << 25, nb=1 << 30: S.lib.spatten_prompt_attention(C.byref(a), ws, nb, None)
    for over, want in [(dict(B=0), S.E_ARG), (dict(B=65536), S.E_ARG), (dict(H=0), S.E_ARG), (dict(H_kv=0), S.E_ARG),
                       (dict(H_kv=3), S.E_SHAPE), (dict(d_h=96), S.E_UNSUPPORTED), (dict(total_q=-1), S.E_ARG),
                       (dict(cu_q=None), S.E_ARG), (dict(cu_kv=None), S.E_SHAPE), (dict(q=None), S.E_ARG),
                       (dict(k=None), S.E_ARG), (dict(v=None), S.E_ARG), (dict(o=None), S.E_ARG), (dict(dtype=2), S.E_ARG),
                       (dict(q_ld_tok=511), S.E_SHAPE), (dict(kv_ld_tok=120), S.E_SHAPE), (dict(o_ld_tok=8), S.E_SHAPE),
                       (dict(weight_cap=0), S.E_SHAPE), (dict(weight_cap=129), S.E_SHAPE),
                       (dict(q=(1 << 20) + 8), S.E_ALIGN), (dict(q_ld_tok=516), S.E_ALIGN), (dict(kv_ld_tok=132), S.E_ALIGN),
                       (dict(o=(1 << 23) + 2), S.E_ALIGN), (dict(kernel=3), S.E_ARG), (dict(kernel=9), S.E_ARG),
                       (dict(kernel=2, dtype=S.F32), S.E_UNSUPPORTED)]:
        assert call(_prompt(S, **over)) == want, over
    assert S.lib.spatten_prompt_attention(None, None, 0, None) == S.E_ARG
    need = S.prompt_workspace_size(_prompt(S))
    assert need >= 8 * 100 * 8                       # two floats per (head, row)
    assert call(_prompt(S), 1 << 25, need - 1) == S.E_WORKSPACE
    assert call(_prompt(S), None, need) == S.E_WORKSPACE
    assert call(_prompt(S), (1 << 25) + 8, need) == S.E_ALIGN
    assert S.prompt_workspace_size(_prompt(S, weight=None)) == 0
    assert call(_prompt(S, total_q=0, total_kv=0, weight=None), None, 0) == S.OK      # nothing to do


def _cache(S, **over):
    c = S.kv4_cache(2, 4, 64, 100, 1 << 20, 1 << 21, 1 << 22, 1 << 23, 1 << 24, 1 << 25)
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(B=0), "E_ARG"), (dict(H_kv=0), "E_ARG"), (dict(cap=0), "E_ARG"), (dict(d_h=32), "E_UNSUPPORTED"),
              (dict(k_codes=None), "E_ARG"), (dict(v_scale=None), "E_ARG"), (dict(k_codes=(1 << 20) + 8), "E_ALIGN"),
              (dict(k_scale=(1 << 21) + 2), "E_ALIGN"), (dict(pos=(1 << 25) + 4), "E_ALIGN")]


def test_append_and_read_refusals(S):
    def append(c=None, k=16, v=32, dt=None, ld=256, total=2, cu=None, ln=48, lo=48, seen=64, so=64):
        return S.lib.spatten_kv4_append(C.byref(c or _cache(S)), k, v, S.BF16 if dt is None else dt, ld, total, cu, ln, lo,
                                        seen, so, None, None)
    for over, want in BAD_CACHES:
        assert append(_cache(S, **over)) == getattr(S, want), over
    assert S.lib.spatten_kv4_append(None, 16, 32, 1, 256, 2, None, 48, 48, 64, 64, None, None) == S.E_ARG
    for over, want in [(dict(k=None), S.E_ARG), (dict(v=None), S.E_ARG), (dict(ln=None), S.E_ARG), (dict(lo=None), S.E_ARG),
                       (dict(dt=2), S.E_ARG), (dict(total=-1), S.E_ARG), (dict(total=3), S.E_SHAPE),
                       (dict(seen=None, so=None), S.E_ARG), (dict(so=None), S.E_ARG), (dict(ld=255), S.E_SHAPE),
                       (dict(k=24), S.E_ALIGN), (dict(ld=260), S.E_ALIGN)]:
        assert append(**over) == want, over
    assert append(_cache(S, pos=None), seen=None) == S.E_ARG       # one of the pair

    def read(c=None, cu=16, row0=None, total=3, ko=32, vo=48, dt=None, ld=256):
        return S.lib.spatten_kv4_read(C.byref(c or _cache(S)), cu, row0, total, ko, vo, S.BF16 if dt is None else dt, ld,
                                      None, None)
    for over, want in BAD_CACHES:
        assert read(_cache(S, **over)) == getattr(S, want), over
    for over, want in [(dict(cu=None), S.E_ARG), (dict(ko=None, vo=None), S.E_ARG), (dict(total=-1), S.E_ARG),
                       (dict(dt=5), S.E_ARG), (dict(ld=100), S.E_SHAPE), (dict(vo=40), S.E_ALIGN), (dict(ld=260), S.E_ALIGN),
                       (dict(total=0), S.OK)]:
        assert read(**over) == want, over


def test_attention_refusals(S):
    def args(c=None, **over):
        a = S.kv4_attn_args()
        a.cache, a.H, a.q, a.dtype, a.q_ld, a.o, a.o_ld = c or _cache(S), 8, 1 << 12, S.BF16, 512, 1 << 13, 512
        a.len, a.n_max, a.update_weight = 1 << 14, 100, 1
        for k, v in over.items():
            setattr(a, k, v)
        return a
    call = lambda a, ws=1 << 26, nb=1 << 30: S.lib.spatten_kv4_attention(C.byref(a), ws, nb, None)
    for over, want in BAD_CACHES:
        assert call(args(_cache(S, **over))) == getattr(S, want), over
    for over, want in [(dict(H=0), S.E_ARG), (dict(H=6), S.E_SHAPE), (dict(q=None), S.E_ARG), (dict(o=None), S.E_ARG),
                       (dict(len=None), S.E_ARG), (dict(dtype=2), S.E_ARG), (dict(n_max=0), S.E_ARG),
                       (dict(n_max=101), S.E_SHAPE), (dict(q_ld=511), S.E_SHAPE), (dict(o_ld=8), S.E_SHAPE),
                       (dict(q=(1 << 12) + 8), S.E_ALIGN), (dict(o_ld=516), S.E_ALIGN)]:
        assert call(args(**over)) == want, over
    assert call(args(_cache(S, weight=None))) == S.E_ARG           # nothing to update
    assert S.lib.spatten_kv4_attention(None, None, 0, None) == S.E_ARG
    need = S.kv4_attention_workspace_size(args())
    assert need > 0
    assert call(args(), 1 << 26, need - 1) == S.E_WORKSPACE and call(args(), None, need) == S.E_WORKSPACE
    assert call(args(), (1 << 26) + 8, need) == S.E_ALIGN


def test_evict_refusals(S):
    def evict(src=None, dst=None, ln=16, lo=16, seen=32, n_max=100, keep=50, recent=10, ws=1 << 26, nb=1 << 30):
        return S.lib.spatten_kv4_evict(C.byref(src or _cache(S)), C.byref(dst or _cache(S)), ln, lo, seen, n_max, keep,
                                       recent, ws, nb, None, None)
    for over, want in BAD_CACHES:
        assert evict(_cache(S, **over)) == getattr(S, want), over
        assert evict(dst=_cache(S, **over)) == getattr(S, want), over
    apart = dict(k_codes=1 << 27, k_scale=1 << 28, v_codes=1 << 29, v_scale=1 << 30, weight=1 << 31, pos=1 << 32)
    for over, want in [(dict(ln=None), S.E_ARG), (dict(lo=None), S.E_ARG), (dict(n_max=0), S.E_ARG), (dict(n_max=101), S.E_SHAPE),
                       (dict(keep=0), S.E_ARG), (dict(recent=-1), S.E_ARG), (dict(recent=51), S.E_ARG),
                       (dict(seen=None), S.E_ARG), (dict(ws=None), S.E_WORKSPACE), (dict(nb=64), S.E_WORKSPACE),
                       (dict(ws=(1 << 26) + 4), S.E_ALIGN), (dict(src=_cache(S, weight=None)), S.E_ARG),
                       (dict(dst=_cache(S, weight=None)), S.E_ARG), (dict(src=_cache(S, pos=None)), S.E_ARG),
                       (dict(dst=_cache(S, B=3)), S.E_SHAPE), (dict(dst=_cache(S, d_h=128)), S.E_SHAPE),
                       (dict(dst=_cache(S, k_codes=1 << 27)), S.E_ARG),            # shares some of src's buffers
                       (dict(dst=_cache(S, cap=60)), S.E_ARG),
                       (dict(dst=_cache(S, cap=49, **apart)), S.E_SHAPE)]:
        assert evict(**over) == want, over
    size = S.kv4_evict_workspace_size
    assert size(_cache(S), 100, 50) >= 8 * 4 * (50 + 50)
    assert size(_cache(S), 0, 50) == 0 and size(_cache(S), 100, 0) == 0


def test_binding_checks_tensors(S):
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    a = S.make_prompt_args(q, k, k, q, cu, weight=torch.zeros(1, 2, 5))
    assert (a.B, a.H, a.H_kv, a.total_q, a.q_ld_tok, a.kv_ld_tok, a.weight_cap, a.dtype) == (1, 4, 2, 5, 256, 128, 5, S.F32)
    with pytest.raises(ValueError):
        S.make_prompt_args(q.transpose(0, 1), k, k, q, cu)
    with pytest.raises(ValueError):
        S.make_prompt_args(q, k, k[:4], q, cu)
    with pytest.raises(TypeError):
        S.make_prompt_args(q, k.bfloat16(), k, q, cu)
    with pytest.raises(TypeError):
        S.make_prompt_args(q, k, k, q, cu.long())
    with pytest.raises(TypeError):
        S.make_prompt_args(q, k, k, q, cu, weight=torch.zeros(1, 4, 5))
    codes, scale = torch.zeros(1, 2, 7, 32, dtype=torch.uint8), torch.zeros(1, 2, 7, 2, dtype=torch.bfloat16)
    c = S.make_kv4_cache(codes, scale, codes, scale, torch.zeros(1, 2, 7))
    assert (c.B, c.H_kv, c.d_h, c.cap, c.pos) == (1, 2, 64, 7, None)
    with pytest.raises(TypeError):
        S.make_kv4_cache(codes, scale.half(), codes, scale)
    with pytest.raises(TypeError):
        S.make_kv4_cache(codes, scale, codes, scale, torch.zeros(1, 2, 8))
    row = torch.zeros(1, 4, 64)
    assert S.make_kv4_attn_args(c, row, row, cu[:1], 7).H == 4
    with pytest.raises(ValueError):
        S.make_kv4_attn_args(c, row[:, :, :32], row, cu[:1], 7)
    with pytest.raises(ValueError):
        S.make_kv4_attn_args(c, row, row, cu, 7)


def test_host_tensors_are_refused(S):
    """Tensors in host memory describe a call, but the call itself refuses them."""
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    cu, n = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        S.prompt_attention(S.make_prompt_args(q, k, k, q, cu))
    codes, scale, w = torch.zeros(1, 2, 7, 32, dtype=torch.uint8), torch.zeros(1, 2, 7, 2, dtype=torch.bfloat16), torch.zeros(1, 2, 7)
    c = S.make_kv4_cache(codes, scale, codes, scale, w)
    with pytest.raises(ValueError):
        S.kv4_append(c, k, k, 128, 5, n, n, cu=cu)
    with pytest.raises(ValueError):
        S.kv4_read(c, cu, 5, k, k, 128)
    with pytest.raises(ValueError):
        S.kv4_attention(S.make_kv4_attn_args(c, q[:1], q[:1], n, 7), w, 28)
    with pytest.raises(ValueError):
        S.kv4_evict(c, c, n, n, None, 7, 3, 0, w, 28)


# ---- the plain forms --------------------------------------------------------------------------------
def test_plain_quantizer_by_hand():
    x = np.zeros(64, np.float32)
    x[:4] = [7.0, -3.5, 0.5, 1.5]            # s = 1; halves round to even
    x[32:34] = [14.0, -1.0]                  # s = 2
    code, s = R.quantize4(x)
    assert s.tolist() == [1.0, 2.0] and code[:4].tolist() == [7, -4, 0, 2] and code[32:34].tolist() == [7, 0]
    assert R.quantize4(np.zeros(32, np.float32))[1].tolist() == [1.0]
    # K: word t*(d/32)+g holds channels 32g+8t..; channel 40 (g=1, t=1, i=0) of 64 is nibble (1*2+1)*8
    one = np.zeros(64, np.int64)
    one[40] = 5
    b = R.pack4(one, 8)
    assert b[12] == 0x88 + 5 and (np.delete(b, 12) == 0x88).all()
    # V: halfword t*(d/32)+g holds channels 32g+4t..; channel 41 (g=1, t=2, i=1) is nibble (2*2+1)*4+1
    one[:] = 0
    one[41] = -3
    b = R.pack4(one, 4)
    assert b[10] == 0x58 and (np.delete(b, 10) == 0x88).all()
    rng = np.random.default_rng(1)
    for d in (64, 128):
        c = rng.integers(-7, 8, (3, d))
        for run in (4, 8):
            assert (R.unpack4(R.pack4(c, run), run) == c).all()


def test_plain_bf16_rounding_matches_torch():
    x = np.random.default_rng(2).standard_normal(4096).astype(np.float32) * np.float32(3e-5)
    np.testing.assert_array_equal(R.to_bf16(x), torch.from_numpy(x).bfloat16().float().numpy())


def test_plain_prompt_matches_torch():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((9, 4, 64)), rng.standard_normal((12, 2, 64)), rng.standard_normal((12, 2, 64))
    o, w = R.prompt_attention(q, k, v, [0, 4, 9], [0, 4, 12], 8)
    for qs, ks in ((slice(0, 4), slice(0, 4)), (slice(4, 9), slice(4, 12))):
        n, m = qs.stop - qs.start, ks.stop - ks.start
        mask = torch.ones(n, m, dtype=torch.bool).tril(m - n)
        t = lambda x: torch.from_numpy(x).transpose(0, 1)[None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            t(q[qs]), t(k[ks]).repeat_interleave(2, 1), t(v[ks]).repeat_interleave(2, 1), attn_mask=mask)
        np.testing.assert_allclose(o[qs], ref[0].transpose(0, 1).numpy(), atol=1e-12)
    assert abs(w[0].sum() - 2 * 2 * 4) < 1e-9 and abs(w[1].sum() - 2 * 2 * 5) < 1e-9


def test_plain_eviction_by_hand():
    w = np.array([5, 1, 4, 4, 9, 2], float)
    assert R.evict_sources(w, None, 6, 0, 3, 0) == [0, 4, 2]          # kept 0, 2, 4: the tie at 4 to row 2
    assert R.evict_sources(w, np.arange(6), 6, 6, 3, 1) == [0, 4, 5]  # row 5 is recent: kept 0, 4, 5
    assert R.evict_sources(w, None, 2, 0, 3, 0) == [0, 1]
    w[0] = np.nan
    assert R.evict_sources(w, None, 6, 0, 3, 0) == [3, 4, 2]
