"""The C ABI of the gated delta rule and of draft verification on the CPU: exports, and every
refusal, all of which come before any HIP call (so no GPU is needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ALIGN, ERR_ALIAS = 0, -1, -2, -3, -4, -5
F32, BF16 = 0, 1
BASE, SPAN = 1 << 40, 1 << 36     # far-apart device addresses that are never touched


@pytest.fixture(scope="module")
def L():
    import rwkv_linear_attention_amd as m
    if not os.path.exists(m.LIB_PATH):
        m.build()
    return m.lib()


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * SPAN + off)


SEQ = ("q", "k", "v", "g", "beta")
DIMS = {"B": 2, "T": 40, "Hk": 2, "H": 4, "K": 64, "V": 128}


def dims(kw):
    return [kw.get(n, DIMS[n]) for n in DIMS]


def forward(L, **kw):
    p = {n: kw.get(n, fake(i)) for i, n in enumerate(SEQ + ("state_in", "o", "state_out"))}
    return L.gdr_forward(*(p[n] for n in SEQ), kw.get("in_dt", BF16), p["state_in"], p["o"], kw.get("o_dt", F32),
                         p["state_out"], kw.get("lengths"), 1.0, *dims(kw), None)


def step(L, **kw):
    p = {n: kw.get(n, fake(i)) for i, n in enumerate(SEQ + ("state_in", "o", "state_out", "state_pos"))}
    return L.gdr_step(*(p[n] for n in SEQ), kw.get("in_dt", BF16), p["state_in"], p["o"], kw.get("o_dt", F32),
                      p["state_out"], p["state_pos"], 1.0, *dims(kw), None)


def ckpt(L, **kw):
    p = {n: kw.get(n, fake(i)) for i, n in enumerate(SEQ + ("state_in", "o", "state_out", "ckpt", "resid"))}
    return L.gdr_forward_ckpt(*(p[n] for n in SEQ), kw.get("in_dt", BF16), p["state_in"], p["o"], p["state_out"],
                              p["ckpt"], p["resid"], 1.0, *dims(kw), None)


BACK = ("q", "k", "g", "beta", "ckpt", "resid", "d_o", "d_state_out", "dq", "dk", "dv", "dg", "dbeta", "d_state_in", "work")


def back(L, **kw):
    p = {n: kw.get(n, fake(i)) for i, n in enumerate(BACK)}
    return L.gdr_backward_ckpt(*(p[n] for n in BACK[:4]), kw.get("in_dt", BF16), *(p[n] for n in BACK[4:]), 1.0,
                               *dims(kw), None)


RUNS = [forward, step, ckpt, back]


def test_every_declared_function_is_exported(L):
    for header in ("gdr.h", "draft.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        names = re.findall(r"^\s*int\s+(\w+)\s*\(", src, flags=re.M)
        assert names
        for n in names:
            assert hasattr(L, n), n


@pytest.mark.parametrize("run", RUNS)
@pytest.mark.parametrize("kw,status", [
    ({"K": 32}, ERR_UNSUPPORTED), ({"K": 96}, ERR_UNSUPPORTED), ({"V": 0}, ERR_UNSUPPORTED),
    ({"V": 100}, ERR_UNSUPPORTED), ({"V": -64}, ERR_UNSUPPORTED), ({"V": 576}, ERR_SHAPE), ({"B": 0}, ERR_SHAPE),
    ({"T": -1}, ERR_SHAPE), ({"Hk": 0}, ERR_SHAPE), ({"H": 0}, ERR_SHAPE), ({"Hk": 3}, ERR_SHAPE),
    ({"H": -4}, ERR_SHAPE), ({"Hk": 8}, ERR_SHAPE), ({"in_dt": 2}, ERR_UNSUPPORTED), ({"B": 1 << 22}, ERR_SHAPE),
    ({"H": 1 << 20}, ERR_SHAPE), ({"T": 2147483647}, ERR_SHAPE), ({"q": None}, ERR_NULL), ({"beta": None}, ERR_NULL),
    ({"k": fake(1, 8)}, ERR_ALIGN), ({"g": fake(3, 4)}, ERR_ALIGN)])
def test_shapes_types_and_pointers(L, run, kw, status):
    assert run(L, **kw) == status


@pytest.mark.parametrize("run", [forward, step])
def test_unknown_output_type(L, run):
    assert run(L, o_dt=3) == ERR_UNSUPPORTED


@pytest.mark.parametrize("run", RUNS[:3])
@pytest.mark.parametrize("name", SEQ)
def test_outputs_over_inputs(L, run, name):
    assert run(L, o=fake(SEQ.index(name))) == ERR_ALIAS
    assert run(L, state_out=fake(SEQ.index(name), 16)) == ERR_ALIAS


def test_states(L):
    for run in RUNS[:3]:
        assert run(L, state_out=fake(5, 64)) == ERR_ALIAS        # over state_in, but not it
        assert run(L, o=fake(7)) == ERR_ALIAS
        assert run(L, state_out=None, **({"state_pos": None} if run is step else {})) == ERR_NULL
    assert step(L, state_pos=fake(7)) == ERR_ALIAS
    assert forward(L, lengths=fake(12, 2)) == ERR_ALIGN
    assert forward(L, lengths=fake(6, 4)) == ERR_ALIAS
    assert step(L, T=0, state_out=None) == ERR_NULL


def test_training_buffers(L):
    assert ckpt(L, ckpt=None) == ERR_NULL and ckpt(L, resid=None) == ERR_NULL
    assert ckpt(L, ckpt=fake(9)) == ERR_ALIAS and ckpt(L, resid=fake(2)) == ERR_ALIAS
    assert ckpt(L, T=1 << 28) == ERR_SHAPE                         # more blocks than a launch covers
    for n in BACK:
        if n != "d_state_out":
            assert back(L, **{n: None}) == ERR_NULL, n
    outs = ("dq", "dk", "dv", "dg", "dbeta", "d_state_in", "work")
    for n in outs:
        for m in BACK:
            if m != n and (n, m) != ("d_state_in", "d_state_out"):
                assert back(L, **{n: fake(BACK.index(m))}) == ERR_ALIAS, (n, m)
    assert back(L, d_state_in=fake(7, 16)) == ERR_ALIAS            # over d_state_out, but not it


DRAFT = ("target", "draft", "tokens", "n_draft", "u", "u_draw", "out", "kept")


def verify(L, dt=F32, B=3, N=4, vocab=1000, **kw):
    p = {n: kw.get(n, fake(i)) for i, n in enumerate(DRAFT)}
    return L.draft_verify(p["target"], p["draft"], dt, *(p[n] for n in DRAFT[2:]), B, N, vocab, None)


@pytest.mark.parametrize("kw,status", [
    ({"dt": 2}, ERR_UNSUPPORTED), ({"B": 0}, ERR_SHAPE), ({"N": -1}, ERR_SHAPE), ({"N": 1025}, ERR_SHAPE),
    ({"vocab": 0}, ERR_SHAPE), ({"vocab": 1 << 25}, ERR_SHAPE), ({"B": 1 << 23}, ERR_SHAPE),
    ({"target": None}, ERR_NULL), ({"tokens": None}, ERR_NULL), ({"u": None}, ERR_NULL), ({"u_draw": None}, ERR_NULL),
    ({"out": None}, ERR_NULL), ({"kept": None}, ERR_NULL), ({"target": fake(0, 4)}, ERR_ALIGN),
    ({"draft": fake(1, 8)}, ERR_ALIGN), ({"tokens": fake(2, 2)}, ERR_ALIGN), ({"out": fake(6, 1)}, ERR_ALIGN)])
def test_draft_refusals(L, kw, status):
    assert verify(L, **kw) == status


def test_draft_outputs_over_inputs(L):
    for n in DRAFT[:6]:
        for o in ("out", "kept"):
            assert verify(L, **{o: fake(DRAFT.index(n))}) == ERR_ALIAS
    assert verify(L, kept=fake(6, 4)) == ERR_ALIAS
