"""Dropout on the host: the generator of the tests against its published vectors, and the C ABI's refusals (CPU only).

The addresses are made up: a call that got past its checks would launch, so every call here must be refused or be empty."""
import pytest

import dropout_ref as ref
from glu_mlp_gemv_amd import api, counter_dropout

OK, NULLP, SHAPE, ALIGN, ALIAS, LAUNCH, UNSUP, STRIDE, WORKSPACE = range(9)
ARG = 10
BF16, FP16, FP32, E4M3 = range(4)
P = [0x100000000 + i * 0x10000000 for i in range(4)]
FULL = 0xFFFFFFFF


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((FULL,) * 4, (FULL,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, words):
    assert tuple(ref.philox4x32_10(counter, key)) == words


def test_draws_are_the_words_halves():
    d = ref.draws(3, 21, 5 << 32 | 7, 9 << 32 | 11)
    for m, k in ((0, 0), (2, 20), (1, 9), (0, 7)):
        w = ref.philox4x32_10((k // 8, m, 11, 9), (7, 5))[k % 8 // 2]
        assert int(d[m, k]) == (w >> 16 if k % 2 else w & 0xFFFF)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=E4M3), ARG), (dict(dtype=-1), ARG), (dict(drop=-1), ARG), (dict(drop=65537), ARG), (dict(M=-1), SHAPE),
    (dict(K=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(x=None), NULLP), (dict(out=None), NULLP), (dict(ldx=99), STRIDE),
    (dict(ldr=99), STRIDE), (dict(ldo=99), STRIDE), (dict(ldx=1 << 62), STRIDE), (dict(x=P[0] + 1), ALIGN),
    (dict(at=P[3] + 4), ALIGN), (dict(dtype=FP32, out=P[2] + 2), ALIGN), (dict(out=P[0] + 2), ALIAS),
    (dict(out=P[1], ldo=101), ALIAS), (dict(out=P[3]), ALIAS), (dict(M=0), OK), (dict(K=0), OK), (dict(M=0, x=None, out=None), OK),
])
def test_refusals(kw, status):
    k = dict(x=P[0], ldx=100, res=P[1], ldr=100, out=P[2], ldo=100, M=5, K=100, drop=6554, at=P[3], dtype=BF16)
    k.update(kw)
    assert api.library().glu_dropout(k["x"], k["ldx"], k["res"], k["ldr"], k["out"], k["ldo"], k["M"], k["K"], k["drop"], 1,
                                     k["at"], 2, k["dtype"], None) == status


def test_probability():
    assert [counter_dropout.drop_of(p) for p in (0, 0.0, 0.1, 0.5, 1.0, 1)] == [0, 0, 6554, 32768, 65536, 65536]
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            counter_dropout.drop_of(p)
