"""The workspace of linear attention: made for the largest prompts, it has to do for all shorter ones."""
import pytest

from weight_only_int4_w4a16_amd import mixers


def size(T, seqs, H, Dk=128, Dv=128):
    return mixers._library().w4a16_linear_attention_workspace(T, seqs, H, Dk, Dv)


def needed(T, seqs, H, D=128):
    """What a call of T tokens uses: states of its segments, their decays, and the maps of many sequences."""
    L = T * H // 256 if T * H // 256 < 512 else max(512, T * H // 512)
    L = min(max((L + 63) // 64 * 64, 256 if T <= 256 else 128), 4096)
    while T // L > 16384:
        L *= 2
    whole = T // L
    slots = (whole + (whole > 0) if seqs == 1 else 2 * whole) + min(seqs, whole)
    up = lambda x: (x + 15) // 16 * 16   # noqa: E731
    return slots * H * D * D * 4 + up(slots * H * 4) + (up(12 * (seqs + 1)) if seqs > 64 else 0)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 7, 8, 16, 32, 33, 64, 100, 128, 257, 258, 259, 300, 512, 600, 32767])
def test_never_less_for_more_tokens(H):
    every = sorted(list(range(0, 20000)) + [4096 * i + d for i in range(5, 400) for d in (-1, 0, 1)] + [
        2 ** i + d for i in range(20, 31) for d in (-1, 0, 1)] + [2 ** 31 - 65])
    last = {s: 0 for s in (1, 2, 9)}
    for T in every:
        for s in last:
            got = size(T, s, H)
            assert got >= last[s], (T, s)
            assert got >= needed(T, s, H), (T, s)
            last[s] = got


@pytest.mark.parametrize("T,H", [(100, 8), (300, 16), (1032, 32), (5000, 1), (32768, 32), (10 ** 6, 2)])
def test_never_less_for_more_sequences(T, H):
    sizes = [size(T, s, H) for s in range(1, 300)] + [size(T, 16384, H)]
    assert sizes == sorted(sizes)


def test_none_where_none_is_needed():
    """A call of up to 255 tokens in one launch takes no memory."""
    for T in (0, 1, 127, 128, 200, 255):
        for H in (1, 8, 64):
            assert size(T, 1, H) == 0 and size(T, 64, H) == 0
    assert size(-1, 1, 8) == -1 and size(10, 0, 8) == -1
