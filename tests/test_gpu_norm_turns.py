"""Group norm where a unit of threads takes several tokens, as in a training batch: the hand-over of the prefetched
token, the tail where the rows are no multiple of the units, and the sums of dweight and dbias over a unit's tokens,
for every unit shape with 16-byte accesses and without.  Tolerances as in test_gpu_norm.py: the sums' fp32 terms
grow with the square root of the rows, as the sums themselves do.
"""
import pytest
import torch

from test_gpu_norm import MODES, check

pytestmark = pytest.mark.gpu

# group width -> threads of its unit (forward, backward), as the launcher's rule has them
UNITS = {8: (8, 8), 64: (8, 8), 128: (16, 16), 256: (32, 32), 512: (32, 32), 1024: (128, 128), 2048: (128, 256),
         4096: (256, 256), 8192: (512, 512), 12000: (512, 512),
         5: (8, 8), 63: (8, 8), 127: (16, 16), 250: (32, 32), 511: (64, 64), 1023: (128, 128), 2047: (256, 256),
         3999: (256, 256), 7001: (512, 512), 11001: (512, 512)}


@pytest.mark.parametrize("D", UNITS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_units_of_several_tokens(dtype, D):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    fwd, bwd = UNITS[D]
    units = sms * 32 * 32 // fwd                       # of one group: 32 warps an SM, in the backward 16
    groups = max(1, units // 160)
    per_group = units // groups
    rows = 5 * per_group // 2 + 1
    assert rows > 2 * per_group and rows % per_group and rows > 4 * (sms * 16 * 32 // bwd // groups)
    i = list(UNITS).index(D) + (dtype == "f32")
    check(dtype, (rows,), groups * D, groups, MODES[i % 4], i % 3 != 0, seed=D)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 63, 512, 2048])
def test_modes_over_several_tokens(mode, D):
    check("bf16", (3, 331), 8 * D if D < 500 else D, 8 if D < 500 else 1, mode, D % 2 == 0, seed=D + 1)


def test_few_channels_of_many_rows():
    # one group of one head's width: hardly more than a token a unit, and the sums are over thousands of units
    check("bf16", (20001,), 128, 1, "gate", False, seed=7)
    check("f32", (20001,), 24, 1, "plain", True, seed=8)
