"""Which kernels the block-scaled FP8 linear runs at which sizes: the shapes on
which the GPU tests check each form are asserted here to select it, so that a
change of the estimates cannot leave a form untested."""
import pytest

import block_scaled_fp4_sigmoid_gb300 as fm
from block_scaled_fp4_sigmoid_gb300 import build

# (T, K, N); K of an odd number of 128-column blocks, with a partial last block and odd N among them
FORMS = {
    "stream 1x2x4": [(1, 16, 1), (3, 1424, 2431), (8, 7168, 576)],
    "stream 1x2x4 ahead": [(8, 1040, 2500), (1, 640, 4703), (5, 144, 2433)],
    "stream 1x3x2 ahead": [(8, 1040, 5003), (1, 400, 9731), (5, 1424, 5003), (3, 144, 5001), (8, 7168, 7168)],
    "stream 1x4x1 ahead": [(7, 1040, 8001), (8, 272, 7301), (1, 656, 9700), (2, 2064, 7999)],
    "stream 2x1x4 ahead": [(16, 2048, 272), (9, 2704, 2333), (128, 656, 129)],
    "stream 2x3x2 ahead": [(16, 1040, 4001), (9, 272, 2500)],
    "tensor 128": [(300, 512, 769), (100, 144, 2000)],
    "tensor 128 split 2": [(513, 2704, 1200)],
    "tensor 128 split 4": [(60, 2064, 2333)],
    "tensor 128 split 8": [(40, 14336, 291), (140, 2704, 300)],
    "tensor 256": [(1030, 1040, 7101)],
    "tensor 256 + 128": [(1024, 1024, 7168), (1000, 1040, 7011)],
}
# (T, H, I): the products of a chain, [T, H] -> 2I -> H
CHAINS = {(7, 2560, 2560): "stream 1x3x2 ahead", (8, 2560, 3968): "stream 1x4x1 ahead"}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_library()


@pytest.mark.parametrize("form,shape", [(f, s) for f, v in FORMS.items() for s in v], ids=str)
def test_the_tested_shapes_select_their_form(form, shape):
    assert fm.linear_fp8_block_form(*shape) == form


def test_the_chains_select_their_forms():
    for (T, H, I), form in CHAINS.items():
        assert fm.linear_fp8_block_form(T, H, 2 * I) == form
        assert fm.linear_fp8_block_form(T, I, H) == "stream 1x2x4 ahead"


def test_no_other_form_exists():
    seen = {fm.linear_fp8_block_form(T, K, N) for T in (1, 2, 7, 8, 9, 16, 17, 40, 64, 128, 129, 200, 513, 1024, 2961, 16384)
            for K in (16, 144, 512, 1024, 2064, 7168, 18432) for N in (1, 300, 576, 1200, 2112, 4800, 5003, 7168, 8001, 36864)}
    assert seen == set(FORMS)


def test_sizes_without_kernels():
    assert fm.linear_fp8_block_form(0, 256, 128) == "none"
    for s in ((-1, 256, 128), (1, 24, 128), (1, 256, 0), (1 << 21, 256, 128)):
        assert fm.linear_fp8_block_form(*s) == "unsupported"
