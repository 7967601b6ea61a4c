"""Rows that begin anywhere in a 16-byte word, the kernels' arithmetic of words restated: what a
warp reads and writes of a piece of 256 elements (no GPU needed)."""
import pytest


def put(base, piece, H, values):
    """Elements written for a row that begins at element `base`: {address: value}, by rw_put."""
    shift = base & 7
    start = 8 - shift
    c0, c1 = piece * 256, min(H, piece * 256 + 256)
    written = {}

    def store(at, v):
        assert at not in written
        written[at] = v

    own = [[values.get(piece * 256 + lane * 8 + i) for i in range(8)] for lane in range(32)]
    for lane in range(32):
        c = (piece * 32 + lane) * 8
        x = (own[lane - 1] if lane else own[0]) + own[lane]     # 16 elements as 8 words of two
        words = [tuple(x[2 * i:2 * i + 2]) for i in range(8)]
        for d in (4, 2, 1):
            if start // 2 & d:
                for i in range(8 - d):
                    words[i] = words[i + d]
        flat = [e for w in words[:5] for e in w]
        g = flat[1:9] if start & 1 else flat[:8]
        word = base + c - shift
        assert word % 8 == 0
        if c - shift >= c0 and c - shift + 8 <= c1:
            for i in range(8):
                store(word + i, g[i])
    head = min(start, c1 - c0) if shift else 0
    tail = min((c1 + shift) & 7, c1 - c0 - head)
    for lane in range(16):
        e = lane if lane < 8 else c1 - c0 - tail + lane - 8
        if lane < head if lane < 8 else lane < 8 + tail:
            assert 0 <= e < 256
            store(base + c0 + e, own[e >> 3][e & 7])
    return written


def read(base, piece, H):
    """Lane's elements as addresses (None: zero), and all addresses read, by copy and read."""
    shift = base & 7
    slot, touched = [None] * (33 * 8), set()
    for lane in range(32):
        c = (piece * 32 + lane) * 8
        word, left = base + c - shift, H - (c - shift)
        own = max(0, min(8, left))
        for i in range(own):
            slot[lane * 8 + i] = word + i
            touched.add(word + i)
        if lane == 31:
            for i in range(max(0, min(shift, left - 8))):
                slot[256 + i] = word + 8 + i
                touched.add(word + 8 + i)
    lanes = []
    for lane in range(32):
        first = (shift >> 1) * 2 + lane * 8        # five words of two
        assert first + 10 <= 33 * 8
        x = slot[first:first + 10]
        lanes.append(x[1:9] if shift & 1 else x[:8])
    return lanes, touched


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 15, 16, 17, 247, 248, 249, 250, 255, 256, 257, 263, 264, 265, 300, 511, 512, 513, 1001])
def test_a_row_is_written_once_and_nothing_else(shift, H):
    base = 800 + shift
    values = {c: ("v", c) for c in range(H)}
    all_written = {}
    for piece in range((H + 255) // 256):
        w = put(base, piece, H, values)
        assert not set(w) & set(all_written)
        all_written.update(w)
    assert all_written == {base + c: ("v", c) for c in range(H)}


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 15, 16, 17, 247, 248, 249, 250, 255, 256, 257, 263, 264, 265, 300, 511, 512, 513, 1001])
def test_a_row_is_read_in_its_words(shift, H):
    base = 800 + shift
    for piece in range((H + 255) // 256):
        lanes, touched = read(base, piece, H)
        for lane in range(32):
            for i in range(8):
                c = (piece * 32 + lane) * 8 + i
                if c < H:
                    assert lanes[lane][i] == base + c
        # nothing behind the row, and before it only what shares its first element's word
        assert all((base & ~7) <= a < base + H for a in touched)
