"""KV4State's host side: what it refuses, before anything of the call has run, and what it holds.  The calls
themselves are replaced and recorded, so a state in host memory will do."""
import pytest
import torch

B, H, HK, D, CAP = 2, 4, 2, 64, 16


@pytest.fixture()
def made(monkeypatch):
    """The module and the list of the library calls made."""
    from cascade_token_head_b200 import build
    build.build()
    from cascade_token_head_b200 import kv4, spatten
    names = []
    monkeypatch.setattr(spatten, "_run", lambda fn, name, *a: names.append(name[len("spatten_"):]))
    return kv4, names


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def rows(n, h, dt=torch.float32):
    return torch.zeros(n, h, D, dtype=dt)


PROMPT = dict(q=rows(5, H), k=rows(5, HK), v=rows(5, HK), cu=i32(0, 2, 5))
RESUME = dict(PROMPT, cu_kv=i32(0, 4, 9), rows=9)
STEP = dict(q=rows(B, H), k=rows(B, HK), v=rows(B, HK))
SHIFTED = torch.zeros(5 * H * D + 2)[2:].view(5, H, D)   # at 8 bytes
BAD_Q = [dict(q=rows(5, H, torch.bfloat16)), dict(q=rows(5, 3)), dict(q=rows(5, H).half()), dict(q=rows(5, H)[:, :, :32]),
         dict(q=SHIFTED), dict(q=rows(1, H).expand(5, H, D)), dict(o=rows(4, H)), dict(o=rows(5, H, torch.bfloat16)), dict(o=SHIFTED)]
BAD = [("prompt", PROMPT, over) for over in BAD_Q + [dict(q=rows(4, H)), dict(cu=i32(0, 5)), dict(cu=i32(0, 2, 5).long()), dict(cu=None)]]
BAD += [("resume", RESUME, over) for over in BAD_Q[1:] + [dict(cu=i32(0, 5)), dict(cu_kv=i32(0, 9)), dict(cu_kv=i32(0, 4, 9).long()),
                                                      dict(cu_kv=None), dict(cu_kv=None, rows=5), dict(rows=-1)]]
BAD += [("step", STEP, over) for over in [dict(q=rows(3, H)), dict(q=rows(B, 3)), dict(q=rows(B, H).half()), dict(o=rows(B, H, torch.bfloat16)),
                                          dict(q=SHIFTED[:B]), dict(o=SHIFTED[:B]), dict(n_max=0), dict(n_max=CAP + 1)]]


@pytest.mark.parametrize("name,args,over", BAD)
def test_a_refused_call_leaves_the_state_as_it_was(made, name, args, over):
    kv4, calls = made
    st = kv4.KV4State(B, H, HK, D, CAP, device="cpu")
    with pytest.raises((TypeError, ValueError, RuntimeError, AttributeError)):
        getattr(st, name)(**dict(args, **over))
    assert calls == [], "rows were appended"


@pytest.mark.parametrize("name,args,want", [
    ("prompt", PROMPT, ["kv4_append", "prompt_attention"]), ("resume", RESUME, ["kv4_append", "kv4_read", "prompt_attention"]),
    ("step", STEP, ["kv4_append", "kv4_attention"]), ("prompt", dict(q=rows(0, H), k=rows(0, HK), v=rows(0, HK), cu=i32(0, 0, 0)),
                                                      ["kv4_append", "prompt_attention"])])
def test_sound_calls_run_in_their_order(made, name, args, want):
    kv4, calls = made
    getattr(kv4.KV4State(B, H, HK, D, CAP, device="cpu"), name)(**args)
    assert calls == want


@pytest.mark.parametrize("h,hk,d", [(3, 2, 64), (0, 1, 64), (1026, 2, 64), (4, 2, 96)])
def test_a_state_that_no_attention_takes_is_refused(made, h, hk, d):
    kv4, _ = made
    with pytest.raises(ValueError):
        kv4.KV4State(B, h, hk, d, CAP, device="cpu")


def test_workspaces_of_a_growing_history_stay_bounded(made):
    """Turn after turn of resume() needs a little more workspace: all that is held stays below four times the
    largest need, and what an earlier call was given stays where it is."""
    kv4, _ = made
    st = kv4.KV4State(1, H, HK, D, 4096, device="cpu")
    given = []
    ask = st._workspace
    st._workspace = lambda key, nb: (given.append((ask(key, nb), nb)), given[-1][0])[1]
    for n in range(20, 4000, 20):
        st.resume(rows(20, H), rows(20, HK), rows(20, HK), i32(0, 20), i32(0, n), n)
    need = max(nb for _, nb in given)
    assert all(ws.numel() >= nb for ws, nb in given) and len({nb for _, nb in given}) > 100
    held = [w for ws in st._ws.values() for w in ws]
    assert sum(w.numel() for w in held) <= 4 * need
    assert {w.data_ptr() for w, _ in given} == {w.data_ptr() for w in held}
