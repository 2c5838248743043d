"""What the serving calls' binding refuses before anything reaches the GPU.  Tensors that claim to be on a GPU
stand in for device ones, and the call itself is replaced: nothing is launched, here or on a GPU machine."""
import pytest
import torch


@pytest.fixture()
def S(monkeypatch):
    from cascade_token_head_b200 import build
    build.build()
    from cascade_token_head_b200 import spatten
    spatten.calls = []
    monkeypatch.setattr(spatten, "_run", lambda fn, name, *a: spatten.calls.append(name))
    yield spatten
    del spatten.calls


class OnGpu(torch.Tensor):
    def get_device(self):
        return 0


def gpu(t):
    return t.as_subclass(OnGpu)


def zeros(*shape, dt=torch.float32):
    return gpu(torch.zeros(shape, dtype=dt))


def i32(*v):
    return gpu(torch.tensor(v, dtype=torch.int32))


B, HK, D, CAP = 2, 2, 64, 9


def cache(S, place=zeros):
    codes = lambda: place(B, HK, CAP, D // 2, dt=torch.uint8)
    scale = lambda: place(B, HK, CAP, D // 32, dt=torch.bfloat16)
    return S.make_kv4_cache(codes(), scale(), codes(), scale(), place(B, HK, CAP), place(B, HK, CAP, dt=torch.int32))


def calls(S):
    """name -> (a call of that operator, its arguments by name)"""
    c, other = cache(S), cache(S)
    q, k = zeros(5, 4, D), zeros(5, HK, D)
    row, ws = zeros(B, 4, D), zeros(1 << 16, dt=torch.uint8)
    prompt = S.make_prompt_args(q, k, k, q, i32(0, 2, 5))
    attend = S.make_kv4_attn_args(c, row, row, i32(3, 3), CAP)
    return {
        "append": (lambda **a: S.kv4_append(c, ld_tok=HK * D, total=5, **a),
                   dict(k=k, v=k, len=i32(0, 0), len_out=i32(0, 0), seen=i32(0, 0), seen_out=i32(0, 0), cu=i32(0, 2, 5), dev_status=i32(0))),
        "read": (lambda **a: S.kv4_read(c, total=5, ld_tok=HK * D, **a),
                 dict(cu=i32(0, 2, 5), k_out=k, v_out=k, row0=i32(0, 0), dev_status=i32(0))),
        "evict": (lambda **a: S.kv4_evict(c, other, n_max=CAP, keep=4, recent=1, ws_bytes=1 << 16, **a),
                  dict(len=i32(0, 0), len_out=i32(0, 0), seen=i32(0, 0), ws=ws, dev_status=i32(0))),
        "prompt": (lambda **a: S.prompt_attention(prompt, ws_bytes=1 << 16, **a), dict(ws=ws)),
        "attend": (lambda **a: S.kv4_attention(attend, ws_bytes=1 << 16, **a), dict(ws=ws)),
    }


OPS = ["append", "read", "evict", "prompt", "attend"]


@pytest.mark.parametrize("op", OPS)
def test_sound_arguments_are_passed_on(S, op):
    call, args = calls(S)[op]
    call(**args)
    assert len(S.calls) == 1


@pytest.mark.parametrize("op", OPS)
def test_host_tensors_next_to_a_cache_on_the_gpu_are_refused(S, op):
    call, args = calls(S)[op]
    for name, t in args.items():
        with pytest.raises(ValueError, match="one device"):
            call(**dict(args, **{name: t.as_subclass(torch.Tensor)}))
    assert not S.calls


def test_eviction_into_a_cache_elsewhere_is_refused(S):
    src, dst = cache(S), cache(S, lambda *shape, dt=torch.float32: torch.zeros(shape, dtype=dt))
    with pytest.raises(ValueError, match="one device"):
        S.kv4_evict(src, dst, i32(0, 0), i32(0, 0), i32(0, 0), CAP, 4, 1, zeros(1 << 16, dt=torch.uint8), 1 << 16)
    assert not S.calls


@pytest.mark.parametrize("op", ["append", "read", "evict"])
def test_counts_and_offsets_are_int32_vectors_of_their_length(S, op):
    """What a kernel reads as B (offsets: B + 1) 32-bit words is that: not int64, not one entry less, not strided.
    What lies behind them is not read."""
    call, args = calls(S)[op]
    for name, t in args.items():
        if t.dtype != torch.int32:
            continue
        n = 1 if name == "dev_status" else (B + 1 if name == "cu" else B)
        with pytest.raises(TypeError):
            call(**dict(args, **{name: zeros(n, dt=torch.int64)}))
        with pytest.raises(TypeError):
            call(**dict(args, **{name: zeros(n)}))
        if n > 1:
            with pytest.raises(TypeError):
                call(**dict(args, **{name: zeros(n, 2, dt=torch.int32)[:, 0]}))
        with pytest.raises(ValueError):
            call(**dict(args, **{name: zeros(n - 1, dt=torch.int32)}))
    assert not S.calls
    call(**{name: zeros(9, dt=torch.int32) if t.dtype == torch.int32 else t for name, t in args.items()})
    assert len(S.calls) == 1


@pytest.mark.parametrize("op,names", [("append", ("k", "v")), ("read", ("k_out", "v_out"))])
def test_row_blocks_of_two_dtypes_are_refused(S, op, names):
    """The wider type's reads or writes would leave the other block."""
    call, args = calls(S)[op]
    for name in names:
        with pytest.raises(TypeError):
            call(**dict(args, **{name: zeros(5, HK, D, dt=torch.bfloat16)}))
        with pytest.raises(TypeError):
            call(**dict(args, **{name: zeros(5, HK, D, dt=torch.float16)}))
    with pytest.raises(TypeError):
        call(dtype=S.BF16, **args)
    assert not S.calls
    call(dtype=S.F32, **args)
    call(dtype=S.BF16, **dict(args, **{name: zeros(5, HK, D, dt=torch.int16) for name in names}))   # bits of that type
    assert len(S.calls) == 2
