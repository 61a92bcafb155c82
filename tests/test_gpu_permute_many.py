"""The row operators where a token's row is shared in ways that fewer tokens or slots do not
reach: three or four wavefronts with several pieces per lane (more than 256 tokens of long rows,
with the weights' gradients or more than eight slots), and up to sixteen aligned rows at once."""
import pytest

from gpu_helpers import say
from rows_helpers import TYPES, wide
from test_gpu_permute import check_all, make

pytestmark = pytest.mark.gpu

# tokens, width, slots.  The first five have, with the weights' gradients, 3 wavefronts of 3 pieces
# per lane, 3 of 2, 3 of 3 with one lane in the last, 4 of 2 and 4 of 3; the others ten to sixteen
# slots in one wavefront, four or (256 tokens) nine
SHAPES = [(300, 4288, 12), (300, 2568, 3), (300, 4104, 9), (257, 4096, 2), (260, 5640, 5), (40, 2048, 12),
          (300, 2048, 16), (256, 4288, 10)]


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,d,k", SHAPES)
def test_long_rows_of_many_tokens(T, d, k, type_):
    say(f"permute of many tokens T={T} d={d} k={k} {type_}")
    pos, w, x, r, _ = make(T, d, k, TYPES[type_], True, 0.3)
    check_all("aligned", pos, w, x, r, k)


@pytest.mark.parametrize("type_", list(TYPES))
def test_long_rows_off_alignment(type_):
    say(f"permute of many tokens off alignment {type_}")
    T, d, k = 290, 2570, 10
    pos, w, x, r, _ = make(T, d, k, TYPES[type_], False, 0.1)
    check_all("one element off", pos, w, x, r, k, lay=lambda t: wide(t, 1, 2))
