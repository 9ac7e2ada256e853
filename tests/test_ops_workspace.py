"""The loss's workspace, no GPU: bounded whatever the vocabulary is."""
import pytest

from tensor_adamw_optimizer_amd import _lib as L

MIB = 1 << 20
DTYPES = [(L.APEXW_BF16, 2), (L.APEXW_F32, 4)]


def _bytes(tokens, d_model, vocab, dtype, backward):
    return L.apexw_linear_xent_workspace_bytes(
        L.apexw_linear_xent_shape(tokens, d_model, vocab, 0, -100, dtype, L.APEXW_LOSS_MEAN), backward)


def _rows(tokens, d_model, eb):
    """The tokens' own places: gathered rows and some words each."""
    return tokens * (d_model * eb + 64)


@pytest.mark.parametrize("dtype,eb", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 64, 65, 1000, 8192, 65536, 1 << 20])
def test_forward(dtype, eb, tokens):
    """A pair for 32 classes of a token at most, of 2^30 logits and the last tile's
    columns (8 pairs a token); small ones are split over k, in slabs of less."""
    for vocab in (1, 1000, 2049, 50000, 131072, 131073, 999983, 1 << 20):
        n = _bytes(tokens, 64, vocab, dtype, False)
        assert n <= 256 * MIB + 64 * tokens + _rows(tokens, 64, eb) + 4 * MIB, (vocab, n)


@pytest.mark.parametrize("dtype,eb", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 64, 1000, 8192, 65536, 1 << 20])
def test_backward(dtype, eb, tokens):
    """A piece's p, and dx's sums; those split over k are of small products."""
    for vocab in (1, 1000, 2049, 50000, 131072, 131073, 999983, 1 << 20):
        n = _bytes(tokens, 64, vocab, dtype, True)
        p = max(256 * MIB, tokens * 2048 * eb)
        assert n <= p + tokens * 64 * 4 + _rows(tokens, 64, eb) + 64 * MIB, (vocab, n)
