"""The oracle of the adapters' operators and of dropout against what is known of them: the
generator's published vectors, masks of the asked share, gradients by differences."""

import numpy as np
import pytest
import torch

from oracle import adapters_oracle as AO


@pytest.mark.parametrize("counter,key,words", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_gives_the_published_vectors(counter, key, words):
    assert AO.philox(np.array([counter]), key)[0].tolist() == words


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_masks_keep_the_asked_share(p):
    n = 1 << 20
    kept = AO.keep_mask(n, p, 12345678901234567, 42).mean()
    # binomial: five standard deviations, and the threshold's step
    assert abs(kept - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n) + 2**-17
    a, b = AO.keep_mask(n, p, 1, 2), AO.keep_mask(n, p, 1, 3)
    assert abs((a & b).mean() - (1 - p) ** 2) <= 5 * np.sqrt(1 / n) and not np.array_equal(a, b)


def test_masks_use_all_words_of_seed_and_offset():
    base = AO.keep_mask(4096, 0.5, 7, 9)
    for seed, offset in ((7 + (1 << 40), 9), (7, 9 + (1 << 40)), (8, 9), (7, 10)):
        assert not np.array_equal(base, AO.keep_mask(4096, 0.5, seed, offset))


@pytest.mark.parametrize("p,ids", [(0.0, [0, 1, 1, -1, 0]), (0.3, [1, 0, 5, 1, 1]), (0.3, None)])
def test_gradients_agree_with_differences(p, ids):
    """loss = sum of Y weighted by dY is linear in each operand: differences are exact to rounding."""
    gen = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    M, N, K, ranks, alpha = 5, 7, 16, [3, 2], [4.0, 1.5]
    w, X, dY = rand(N, K), rand(M, K), rand(M, N)
    A, B = [rand(r, K) for r in ranks], [rand(N, r) for r in ranks]
    ids = None if ids is None else torch.tensor(ids)
    loss = lambda: float((AO.fwd(w, A, B, alpha, X, ids, p, (5, 6))["Y"] * dY).sum())  # noqa: E731
    got = AO.bwd(w, A, B, alpha, X, dY, ids, p, (5, 6))
    for t, grad in [(X, got["dX"]), *zip(A, got["dA"]), *zip(B, got["dB"])]:
        flat, g = t.view(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), 5):
            kept = float(flat[i])
            flat[i] = kept + 0.5
            up = loss()
            flat[i] = kept - 0.5
            down = loss()
            flat[i] = kept
            assert abs(up - down - float(g[i])) <= 1e-10 * (1 + abs(float(g[i])))


def test_rows_without_an_adapter_have_the_base_product():
    w, X = torch.randn(6, 8), torch.randn(3, 8)
    A, B = [torch.randn(2, 8)], [torch.randn(6, 2)]
    out = AO.fwd(w, A, B, [2.0], X, torch.tensor([-1, 7, 0]))
    base = X.double() @ w.double().T
    assert torch.equal(out["Y"][:2], base[:2]) and not torch.equal(out["Y"][2], base[2])
    assert not out["T"][:2].any() and not out["T"][:, 2:].any()
