"""Norm and rotation at far positions, on the GPU: the angle is the float64
product of position and frequency, and its sine and cosine are those of that
angle however large it is."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [1 << 20, 1 << 28, 1 << 40, 1 << 52, (1 << 63) - 1])
def test_sines_of_far_positions(far, interleaved):
    # Heads of (1, 0) pairs turn to cosine and sine, rounded to float32 and then to bf16: half a step (2^-8 of the value) and
    # 2^-24, with 2^-40 for the sines themselves (their turns are exact to some 2^-46 at the last of these positions).
    import torch
    import markov_draft_sampling_amd as mds
    T, D = 64, 128
    g = torch.Generator().manual_seed(0)
    pos = torch.cat([torch.randint(far // 2, far, (T - 2,), generator=g), torch.tensor([far, -far])])
    freq, _ = mds.rope_frequencies(D, device="cpu")
    x = torch.zeros((T, 1, D), dtype=torch.bfloat16)
    first = torch.arange(D // 2) * 2 if interleaved else torch.arange(D // 2)
    second = first + 1 if interleaved else first + D // 2
    x[..., first] = 1.0
    q = x.cuda()
    k, qo, ko = q.clone(), torch.zeros_like(q), torch.zeros_like(q)
    mds.qk_norm_rope(q, k, pos.cuda(), freq.cuda(), qo, ko, interleaved=interleaved)
    a = pos.double()[:, None] * freq[None, :]
    for o in (qo, ko):
        o = o.cpu().double()[:, 0]
        for got, want in ((o[:, first], torch.cos(a)), (o[:, second], torch.sin(a))):
            err = (got - want).abs()
            tol = (2.0 ** -8 + 2.0 ** -24) * want.abs() + 2.0 ** -40
            assert (err <= tol).all(), (far, float(err.max()))


def test_codes_of_far_keys_are_those_of_separate_operations():
    # Every float32 factor the nearest to that of the float64 angle: codes of an 8-bit cache equal those of separate
    # operations but where a sine lies within 2^-50 of the middle of two float32s (1 in 10^7) and a code next to a border.
    import torch
    import markov_draft_sampling_amd as mds
    T, Hk, D = 256, 8, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, 2 + 2 * Hk, D), generator=g).to(torch.bfloat16)
    pos = torch.randint(1 << 32, 1 << 40, (T,), generator=g)
    freq, _ = mds.rope_frequencies(D, device="cpu")
    scale = torch.linspace(0.003, 0.03, Hk)
    kp, vp = (torch.zeros((T // 16, 16, Hk, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    d = x.cuda()
    mds.qk_norm_rope_append(d[:, :2], d[:, 2:2 + Hk], d[:, 2 + Hk:], pos.cuda(), freq.cuda(), torch.empty_like(d[:, :2]), kp, vp,
                            torch.arange(T).cuda(), k_scale=scale.cuda(), v_scale=scale.cuda())
    k = x[:, 2:2 + Hk].float()
    a = pos.double()[:, None] * freq
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    p, q = k[..., :D // 2], k[..., D // 2:]
    k = torch.cat([p * c - q * s, q * c + p * s], -1)
    want = (k / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(kp.view(torch.uint8).cpu().view(T, Hk, D), want.view(torch.uint8))
