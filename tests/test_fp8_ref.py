"""The 8-bit path's checks on the host: they pass a result that is right but for its rounding and see planted mistakes."""
import pytest
import torch

import fp8_ref as ref


def operands(M, N, K, mats):
    g = torch.Generator().manual_seed(M + N + K)
    x, sx = ref.quantize32(torch.randn(M, K, generator=g) * torch.exp(torch.randn(K, generator=g) * 0.5), False)
    out = [x, sx]
    for _ in range(mats):
        out += ref.quantize32(torch.randn(N, K, generator=g) * 0.05, True)
    return out


def result(ops):
    y, e = ref.product64(*ops[:4])
    return y if len(ops) == 4 else ref.glu64(y, e, *ref.product64(*ops[:2], *ops[4:]))[0]


@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M,N,K", [(37, 150, 1024), (65, 300, 272)])
def test_root_mean_square_check(M, N, K, mats):
    ops = operands(M, N, K, mats)
    y = result(ops)
    for t in (torch.bfloat16, torch.float16):
        ref.check_unit_rms("rounded", y.to(t), ops)
        # a factor beyond the store's rounding, a lost K-block, one product's scale for the other's
        planted = [y * (1 + 4 * ref.half(t)), y * (1 - 4 * ref.half(t)), result([t_[..., :K - 16] if t_.dtype is ref.E4M3 else t_
                                                                                for t_ in ops])]
        if mats == 2:
            planted.append(result([*ops[:4], ops[4], ops[3]]))
        for wrong in planted:
            with pytest.raises(AssertionError):
                ref.check_unit_rms("planted", wrong.to(t), ops)
