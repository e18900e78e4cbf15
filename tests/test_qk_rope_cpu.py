"""The rotating calls without a GPU: refusals of the C ABI, and the frequencies of
rotary.py against their definitions."""
import ctypes
import math
import shutil
import os

import pytest

from verify_dspark_markov_step_gb300 import rotary


@pytest.fixture(scope="module")
def L():
    if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from verify_dspark_markov_step_gb300 import build, _lib
    build.build()
    return _lib.lib()


FAKE = ctypes.c_void_p(4096)  # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p(4098)


def test_rows_refusals(L):
    def call(q=FAKE, qo=FAKE, k=FAKE, ko=FAKE, dt=1, qs=1024, qos=1024, ks=256, kos=256, pos=FAKE,
             turns=FAKE, factor=1.0, R=64, inter=0, qw=None, kw=None, eps=1e-6, Hq=8, H=2, D=128,
             T=4):
        return L.dspark_qk_rope(q, qo, k, ko, dt, qs, qos, ks, kos, pos, turns, factor, R, inter,
                                qw, kw, eps, Hq, H, D, T, None)
    assert call(T=-1) == -1
    assert call(T=1 << 30) == -1
    assert call(Hq=0) == -1
    assert call(H=-1) == -1
    assert call(H=1025) == -1
    assert call(dt=0) == -1
    assert call(dt=3) == -1
    assert call(D=8) == -2
    assert call(D=120) == -2
    assert call(D=272) == -2
    assert call(R=-16) == -1
    assert call(R=144) == -1
    assert call(R=24) == -2
    assert call(turns=None) == -1
    assert call(turns=ctypes.c_void_p(4100)) == -7
    assert call(factor=math.inf) == -1
    assert call(factor=math.nan) == -1
    assert call(inter=2) == -1
    assert call(qw=FAKE, eps=-1.0) == -1
    assert call(kw=FAKE, eps=math.nan) == -1
    assert call(qw=ODD) == -7
    assert call(q=None) == -1
    assert call(qo=None) == -1
    assert call(k=None) == -1
    assert call(ko=None) == -1
    assert call(pos=None) == -1
    assert call(q=ODD) == -7
    assert call(ko=ODD) == -7
    assert call(qs=1028, qos=1028) == -7
    assert call(ks=-256, kos=-256) == -7
    assert call(qo=FAKE, q=FAKE, qos=2048) == -1      # in place with other strides
    assert call(ko=FAKE, k=FAKE, kos=512) == -1
    assert call(T=0, q=None) == 0


def test_append_refusals(L):
    from verify_dspark_markov_step_gb300 import _lib

    def call(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, dt=1, qs=1024, qos=1024, ks=1024, vs=1024, pos=FAKE,
             slot=FAKE, turns=FAKE, factor=1.0, R=64, inter=0, qw=None, kw=None, eps=1e-6, Hq=8,
             T=4, cache=True, **kw_cache):
        d = dict(k=4096, v=4096, k_scale=None, v_scale=None, k_block_stride=8 * 16 * 128,
                 k_head_stride=16 * 128, k_token_stride=128, v_block_stride=8 * 16 * 128,
                 v_head_stride=16 * 128, v_token_stride=128, dtype=1, num_blocks=10, kv_heads=8,
                 page_size=16, head_dim=128)
        d.update(kw_cache)
        c = _lib.PagedKv(**d) if cache else None
        return L.dspark_qk_rope_append(q, qo, k, v, dt, qs, qos, ks, vs, c, pos, slot, turns,
                                       factor, R, inter, qw, kw, eps, Hq, T, None, None)
    assert call(cache=False) == -1
    assert call(T=-1) == -1
    assert call(Hq=0) == -1
    assert call(dt=2) == -2                # fp16 rows, bf16 cache
    assert call(head_dim=96) == -2
    assert call(page_size=48) == -2
    assert call(R=144) == -1
    assert call(R=40) == -2
    assert call(turns=None) == -1
    assert call(qw=FAKE, eps=math.inf) == -1
    for name in ("q", "qo", "k", "v", "pos", "slot"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "qo", "k", "v"):
        assert call(**{name: ODD}) == -7, name
    for name in ("qs", "qos", "ks", "vs"):
        assert call(**{name: 1028, **({"qos": 1028} if name == "qs" else {"qs": 1028} if name == "qos" else {})}) == -7, name
    assert call(qos=2048) == -1
    assert call(k_token_stride=132) == -7
    assert call(T=0) == 0


def test_binding_refuses_what_is_no_cuda_tensor():
    import torch
    from verify_dspark_markov_step_gb300 import _lib
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        _lib.qk_rope(q, None, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="CUDA"):
        _lib.qk_rope_append(q, q, q, q, q, None, None)


def test_plain_frequencies():
    w, m = rotary.frequencies(64, 5e5)
    assert m == 1.0 and len(w) == 32 and w[0] == 1.0
    for i, x in enumerate(w):
        assert math.isclose(x, math.exp(-2 * i / 64 * math.log(5e5)), rel_tol=1e-13)


def test_linear_and_ntk():
    plain, _ = rotary.frequencies(128)
    w, _ = rotary.frequencies(128, scaling={"type": "linear", "factor": 8})
    assert all(math.isclose(a, b / 8, rel_tol=1e-15) for a, b in zip(w, plain))
    w, _ = rotary.frequencies(128, scaling={"type": "ntk", "factor": 8})
    assert w[0] == plain[0]
    assert math.isclose(w[-1], plain[-1] / 8, rel_tol=1e-12)
    assert all(p / 8 * (1 - 1e-12) <= a <= p for a, p in zip(w, plain))


def test_by_parts():
    s = {"type": "by_parts", "factor": 8, "original_max_position": 8192}
    plain, _ = rotary.frequencies(128, 5e5)
    w, m = rotary.frequencies(128, 5e5, s)
    assert m == 1.0
    kinds = set()
    for a, p in zip(w, plain):
        wavelength = 2 * math.pi / p
        if wavelength < 8192 / 4:
            assert a == p
            kinds.add("kept")
        elif wavelength > 8192:
            assert math.isclose(a, p / 8, rel_tol=1e-15)
            kinds.add("slowed")
        else:
            t = (8192 / wavelength - 1) / 3
            assert math.isclose(a, (1 - t) * p / 8 + t * p, rel_tol=1e-12)
            kinds.add("between")
    assert len(kinds) == 3
    assert all(a > b for a, b in zip(w, w[1:]))


def test_yarn():
    s = {"type": "yarn", "factor": 16, "original_max_position": 8192}
    plain, _ = rotary.frequencies(128, 1e4)
    w, m = rotary.frequencies(128, 1e4, s)
    assert math.isclose(m, 0.1 * math.log(16) + 1)
    turns = [8192 * p / (2 * math.pi) for p in plain]
    for a, p, t in zip(w, plain, turns):
        assert p / 16 * (1 - 1e-12) <= a <= p
        if t > 33:                      # (the ramp's ends are whole pairs)
            assert a == p
        if t < 0.8:
            assert math.isclose(a, p / 16, rel_tol=1e-15)
    assert rotary.frequencies(128, 1e4, {**s, "attention_factor": 1.25})[1] == 1.25
    assert rotary.frequencies(128, 1e4, {**s, "factor": 1})[1] == 1.0


def test_frequencies_refusals():
    for kw in ({"rotary_dim": 0}, {"rotary_dim": 7}, {"rotary_dim": 64, "base": 0.0},
               {"rotary_dim": 64, "base": math.inf},
               {"rotary_dim": 64, "scaling": {"type": "other"}},
               {"rotary_dim": 64, "scaling": {"type": "linear", "factor": 0}},
               {"rotary_dim": 64, "scaling": {"type": "linear", "factor": 2, "slow_turns": 1}},
               {"rotary_dim": 2, "scaling": {"type": "ntk", "factor": 2}},
               {"rotary_dim": 64, "scaling": {"type": "by_parts", "factor": 2, "low_turns": 4,
                                              "original_max_position": 100}},
               {"rotary_dim": 64, "scaling": {"type": "yarn", "factor": 2, "fast_turns": 1,
                                              "original_max_position": 100}}):
        with pytest.raises(ValueError):
            rotary.frequencies(**kw)
    with pytest.raises(KeyError):
        rotary.frequencies(64, scaling={"type": "yarn", "factor": 2})
    with pytest.raises(ValueError):
        rotary.turns_of([math.inf])
    with pytest.raises(ValueError):
        rotary.Rotary(24, device="cpu")
    with pytest.raises(ValueError):
        rotary.Rotary(32, radians=[1.0] * 15, device="cpu")


def test_turns_are_the_frequencies_modulo_a_turn():
    values = [1.0, 0.1, 1e-6, 3.0, 7.0, -0.5, 0.0, 2 * math.pi]
    for w, t in zip(values, rotary.turns_of(values)):
        assert 0 <= t < 2 ** 64
        got = t / 2.0 ** 64
        want = w / (2 * math.pi) % 1.0
        assert min(abs(got - want), 1 - abs(got - want)) <= 2 ** -52
    # one radian to 2^-64 turns: 1 / (2 pi) = 0.15915494309189533577 (rounded after 20 places)
    assert abs(rotary.turns_of([1.0])[0] - 15915494309189533577 * 2 ** 64 // 10 ** 20) <= 1


def test_rotary_holds_signed_words():
    r = rotary.Rotary(32, radians=[3.0 + 0.1 * i for i in range(16)], device="cpu", interleaved=True)
    assert r.turns.shape == (16,)
    back = [t % 2 ** 64 for t in r.turns.tolist()]
    assert back == rotary.turns_of(r.radians)
    assert min(r.turns.tolist()) < 0 < max(r.turns.tolist())
    assert r.args()["interleaved"] is True and r.args()["factor"] == 1.0
