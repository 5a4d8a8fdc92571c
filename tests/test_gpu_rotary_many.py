"""Rotary positions of many tokens, several to a CTA, against the oracle: every width of a unit (pairs in eights, fours, twos and
alone), both layouts and types, in place and beside, rows in use that end inside a CTA's tokens."""
import pytest

import bit_quantized_expert_gb300 as moe
from test_gpu_rotary import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_expert_gb300 import build
    build.build()
    moe.load_library()


@pytest.mark.parametrize("in_place,fused", [(False, False), (True, False), (True, True), (False, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 96), (128, 24), (64, 20), (64, 30), (128, 2), (256, 256), (80, 52), (8, 6)])
def test_many_tokens(D, rot, layout, dtype, in_place, fused):
    run(T=613, Hq=3, Hkv=2, D=D, rot=rot, layout=layout, dtype=dtype, in_place=in_place, fused=fused, seed=rot)


@pytest.mark.parametrize("n_rows", [0, 1, 5, 607, 610, 611, 612, 613, 4000])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 24), ("half", 30), ("interleaved", 48)])
def test_rows_in_use_end_anywhere(layout, rot, n_rows):
    for in_place in (False, True):
        run(T=613, Hq=2, Hkv=1, D=64, rot=rot, layout=layout, n_rows=n_rows, in_place=in_place, dtype="fp16", seed=n_rows)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 8), (5, 0, 64), (0, 7, 128), (32, 8, 128), (1, 1, 256)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_head_counts(Hq, Hkv, D, layout):
    run(T=1217, Hq=Hq, Hkv=Hkv, D=D, rot=D, layout=layout, n_rows=1215, seed=Hq)
