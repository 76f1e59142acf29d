"""Packed tensors of more than 2^32 elements through dropout, whatever shape they
have."""
import numpy as np
import pytest

import map_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def test_dropout_of_more_than_2_to_the_32_elements(rz):
    n = (1 << 32) + 8 * 5 + 3       # a tail past the last whole vector
    flat = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for shape in [(n,), (n, 1), (1, n)]:
        flat.fill_(1.0)
        x = flat.view(shape)
        rz.map_dropout(x, x, 0.5, 31, 32)
        for first, count in ((0, 1024), ((1 << 31) - 512, 1024), ((1 << 32) - 512, 555)):
            want = ref.drop_factor((count,), 0.5, 31, 32, first=first)
            np.testing.assert_array_equal(ref.host(flat[first:first + count]), want)


def test_dropout_of_an_odd_number_past_2_to_the_31(rz):
    n = (1 << 31) + 11
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    r = torch.full((n,), 0.25, dtype=torch.float16, device="cuda")
    rz.map_dropout(x, r, 0.25, 3, 4, residual=r)
    for first, count in ((0, 1024), ((1 << 31) - 512, 523)):
        want = ref.drop_factor((count,), 0.25, 3, 4, first=first)
        # 65536 / 49152 + 1/4 in eleven significant bits: one float32 product, one sum, one rounding
        got = ref.host(r[first:first + count])
        assert np.all(np.abs(got - (want + 0.25)) <= ref.stored(want + 0.25, 3 * ref.U * (want + 0.25), "f16"))
        np.testing.assert_array_equal(got == 0.25, want == 0)
