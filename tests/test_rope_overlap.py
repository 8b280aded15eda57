"""What a rotary call writes must not be what it reads or writes elsewhere: the check of two
strided views (csrc/byte_views.h, compiled alone) against their bytes counted out, and the
calls that it refuses. Runs on the CPU; nothing is launched."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from sparse_window_attention_b200 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("views") / "views_check")
    subprocess.run([gxx, "-std=c++17", "-O2", os.path.join(ROOT, "tests", "native", "views_check.cpp"), "-o", exe], check=True)

    def run(pairs):
        text = "".join(" ".join(str(int(x)) for v in pair for x in (v[0], v[1], *sum(map(tuple, v[2]), ()))) + "\n" for pair in pairs)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(pairs)
        return [x == "1" for x in out]

    return run


def _bytes(view):
    base, row, axes = view
    at = np.array([base])
    for step, ext in axes:
        at = (at[:, None] + step * np.arange(ext)).ravel()
    return set((at[:, None] + np.arange(row)).ravel().tolist())


def test_views_against_their_bytes_counted_out(meet):
    rng = np.random.default_rng(7)
    pairs = []
    for _ in range(3000):
        row = 16 * int(rng.integers(1, 4))
        nested, step = [], row
        for _ in range(3):  # slices of one layout, with gaps
            step *= int(rng.integers(1, 4))
            nested.append([step, int(rng.integers(1, 5))])
            step *= nested[-1][1]
        pair = []
        for _ in range(2):
            axes = [list(a) for a in nested]
            if rng.random() < 0.5:  # another layout: any steps, 0 among them
                axes = [[16 * int(rng.integers(0, 30)), int(rng.integers(1, 5))] for _ in range(3)]
            for a in axes:
                a[1] = int(rng.integers(1, a[1] + 1))
            pair.append((1000 * 16 + 16 * int(rng.integers(0, 40)), row, [axes[i] for i in rng.permutation(3)]))
        pairs.append(pair)
    want = [bool(_bytes(a) & _bytes(b)) for a, b in pairs]
    assert 0.2 < np.mean(want) < 0.8
    assert meet(pairs) == want and meet([(b, a) for a, b in pairs]) == want


def test_slices_of_large_buffers(meet):
    """Packed projections and sequences split into image and text rows, at real sizes: decided
    exactly, in the bounded number of steps."""
    b, n, text, h, d = 2, 32760, 512, 12, 256  # d in bytes
    base = 0x7F0000000000
    packed = lambda slot, rows=n, row0=0, heads=h: (base + slot * h * d + row0 * 3 * h * d, d, [(rows * 3 * h * d if not row0 else n * 3 * h * d, b), (d, heads), (3 * h * d, rows - row0)])  # noqa: E731,E501
    seq = lambda first, rows: (base + first * d, d, [(h * (n + text) * d, b), ((n + text) * d, h), (d, rows)])  # noqa: E731
    cases = [
        (packed(0), packed(1), False), (packed(0), packed(2), False), (packed(1), packed(1), True),
        (seq(0, n), seq(n, text), False), (seq(0, n), seq(n - 1, text), True), (seq(0, n + 1), seq(n, text), True),
        (seq(0, n), (base + (h * (n + text) - 1) * d, d, [(0, 1)] * 3), False),  # the last head's last text row
        (seq(0, n), (base + (h * (n + text) - text - 1) * d, d, [(0, 1)] * 3), True),  # its last image row
        # one record a batch entry: [n, 3, h] rows, then [text, 3, h] rows, of unlike batch strides to a compact copy
        ((base, d, [((n + text) * 3 * h * d, b), (d, h), (3 * h * d, n)]),
         (base + n * 3 * h * d, d, [((n + text) * 3 * h * d, b), (d, h), (3 * h * d, text)]), False),
        ((base, d, [(h * n * d, b), (n * d, h), (d, n)]), (base + b * h * n * d, d, [(h * n * d, b), (n * d, h), (d, n)]), False),
        ((base, d, [(h * n * d, b), (n * d, h), (d, n)]), (base + d * (b * h * n - 1), d, [(3 * h * d, n), (d, h), (0, 1)]), True),
    ]
    assert meet([c[:2] for c in cases]) == [c[2] for c in cases]


FAKE = 0x7F0000000000  # never dereferenced: every call here is refused


def _p():
    return B.make_params(1, 2, 128, (1, 64, 64), (1, 16, 16), (0, 0, 0), (0, 0, 0), 16, 0, "bf16")


ROPE = B.make_rope_params((16, 56, 56))
MB = 1 << 20


def _tensor(x=FAKE, y=FAKE + 32 * MB, dy=FAKE + 64 * MB, weight=None, dweight=None, rows=4096, first=0, strides=None):
    s = strides or (2 * 4112 * 128, 4112 * 128, 128)
    return B.rope_tensor(x, y, 2, rows, first, 1, weight, dy, dweight, strides={"x": s, "y": s, "dy": s})


def _fwd(*t):
    return B.basa_rope_fwd(list(t), FAKE + 512 * MB, 1e-6, ROPE, _p(), stream=0, check=False)


def _bwd(*t):
    return B.basa_rope_bwd(list(t), FAKE + 512 * MB, 1e-6, FAKE + 600 * MB, ROPE, _p(), stream=0, check=False)


def test_overlapping_tensors_are_refused():
    row = 256  # bytes
    y = FAKE + 32 * MB
    # two parts of one sequence that share a row, at different bases
    text = dict(x=FAKE + 128 * MB, dy=FAKE + 160 * MB, rows=16, first=4096)
    assert _fwd(_tensor(), _tensor(y=y + 4095 * row, **text)) == 1
    assert _fwd(_tensor(y=y + 4095 * row, **text), _tensor()) == 1
    assert _bwd(_tensor(), _tensor(y=y + 4095 * row, **text)) == 1
    # an output that starts inside another part's input, or inside its own
    assert _fwd(_tensor(), _tensor(x=y + 100 * row, y=FAKE + 128 * MB)) == 1
    assert _fwd(_tensor(y=FAKE + row)) == 1 and _fwd(_tensor(y=FAKE + 16)) == 1
    assert _bwd(_tensor(y=FAKE + 64 * MB + row)) == 1 and _bwd(_tensor(weight=FAKE + 256 * MB, y=FAKE + row)) == 1
    # gradients and weights
    w, dw = FAKE + 256 * MB, FAKE + 257 * MB
    assert _bwd(_tensor(weight=w, dweight=dw), _tensor(x=FAKE + 128 * MB, y=FAKE + 160 * MB, dy=FAKE + 192 * MB, weight=w, dweight=dw + 128)) == 1
    assert _bwd(_tensor(weight=w, dweight=y + 7 * row)) == 1 and _bwd(_tensor(weight=y + 7 * row, dweight=dw)) == 1
    assert _fwd(_tensor(weight=y + 4095 * row + 16)) == 1
