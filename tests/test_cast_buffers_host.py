"""Without a GPU: the binding of the MX casts, and of their statistics, refuses
tensors that the calls, which take bare pointers, would read or write wrongly or
past their ends."""
import pytest
import torch

from tensor_scaling_cast_gb300 import fp8q as F

ROWS, COLS = 64, 96
FORMATS = [F.E2M1, F.E4M3, F.E5M2]


def new(rows, cols, fmt):
    return F.MXMatrix.allocate(rows, cols, fmt, device="cpu")


def calls(x, m, t, fmt):
    """The casts of x into m and, dual, t."""
    cast = [lambda: F.mx_cast_ex(x, fmt, 0, 0, F.MX_ROWWISE, m.q, m.e8m0),
            lambda: F.mx_cast_dual(x, fmt, 0, 0, m.q, m.e8m0, t.q, t.e8m0),
            lambda: F.mx_cast(x, fmt, 0, m.q, m.e8m0)]
    # the statistics of 8-bit codes read what the casts write
    return cast + ([] if fmt == F.E2M1 else [lambda: F.mx_error_stats(x, m.q, m.e8m0, fmt, torch.zeros(3))])


def columns(m, at, cols):
    """A slice of a wider matrix."""
    per = 2 if m.fmt == F.E2M1 else 1
    return F.MXMatrix(m.q[:, at // per:(at + cols) // per], m.e8m0[:, at // 32:(at + cols) // 32], m.fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_slices_are_refused(fmt):
    x = torch.zeros(ROWS, COLS, dtype=torch.bfloat16)
    part, part_t = columns(new(ROWS, COLS + 64, fmt), 32, COLS), columns(new(COLS, ROWS + 64, fmt), 32, ROWS)
    for call in calls(x, part, new(COLS, ROWS, fmt), fmt):
        with pytest.raises(TypeError, match="contiguous"):
            call()
    m = new(ROWS, COLS, fmt)
    with pytest.raises(TypeError, match="contiguous"):
        F.mx_cast_dual(x, fmt, 0, 0, m.q, m.e8m0, part_t.q, part_t.e8m0)
    wide = torch.zeros(ROWS, 2 * COLS, dtype=torch.bfloat16)
    for bad in (wide[:, :COLS], wide[:, ::2], torch.zeros(COLS, ROWS).t()):
        for call in calls(bad, m, new(COLS, ROWS, fmt), fmt):
            with pytest.raises(TypeError, match="contiguous"):
                call()


@pytest.mark.parametrize("fmt", FORMATS)
def test_buffers_too_short_are_refused(fmt):
    x = torch.zeros(ROWS, COLS, dtype=torch.bfloat16)
    good, good_t = new(ROWS, COLS, fmt), new(COLS, ROWS, fmt)
    for m, t in ((new(ROWS - 1, COLS, fmt), good_t), (good, new(COLS, ROWS - 32, fmt))):
        with pytest.raises(TypeError, match="hold"):
            F.mx_cast_dual(x, fmt, 0, 0, m.q, m.e8m0, t.q, t.e8m0)
    for q, e in ((good.q[:-1], good.e8m0), (good.q, good.e8m0[:-1])):
        for call in (lambda: F.mx_cast_ex(x, fmt, 0, 0, F.MX_ROWWISE, q, e), lambda: F.mx_cast(x, fmt, 0, q, e)):
            with pytest.raises(TypeError, match="hold"):
                call()


def test_codes_of_8_bits_do_not_go_into_a_4_bit_matrix():
    x = torch.zeros(ROWS, COLS)
    four, four_t = new(ROWS, COLS, F.E2M1), new(COLS, ROWS, F.E2M1)
    for call in calls(x, four, four_t, F.E4M3) + [
            lambda: F.mx_cast_ex(x, F.E5M2, 0, 0, F.MX_COLWISE, four.q, four.e8m0)]:
        with pytest.raises(TypeError, match="hold"):
            call()


def test_codes_of_4_bits_go_into_rows_of_their_length():
    x = torch.zeros(ROWS, COLS)
    eight, eight_t, wide = new(ROWS, COLS, F.E4M3), new(COLS, ROWS, F.E4M3), new(ROWS, 2 * COLS, F.E2M1)
    for m in (eight, wide):
        for call in calls(x, m, eight_t, F.E2M1):
            with pytest.raises(TypeError, match="rows of 96"):
                call()
    with pytest.raises(TypeError, match="rows of 64"):
        four = new(ROWS, COLS, F.E2M1)
        F.mx_cast_dual(x, F.E2M1, 0, 0, four.q, four.e8m0, eight_t.q, eight_t.e8m0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_host_memory_is_refused(fmt):
    x = torch.zeros(ROWS, COLS, dtype=torch.bfloat16)
    for call in calls(x, new(ROWS, COLS, fmt), new(COLS, ROWS, fmt), fmt):
        with pytest.raises(TypeError, match="cpu"):
            call()
    # buffers larger than a call needs, or flat ones, are no reason to refuse it
    large = torch.zeros(2 * ROWS, COLS // 2 if fmt == F.E2M1 else COLS, dtype=torch.uint8)
    with pytest.raises(TypeError, match="cpu"):
        F.mx_cast_ex(x, fmt, 0, 0, F.MX_ROWWISE, large, torch.zeros(ROWS * COLS, dtype=torch.uint8))
