"""The machine code of mxq_act_grad's kernels for whole rows: a wave keeps four rows in flight, and
the first row's arithmetic waits for its own loads alone, not for those of the rows behind it."""
import re

import pytest

from tests.test_machine_code_cpu import kernels  # noqa: F401

ROWS = 4


def row_loads(gated: bool, fp32: bool) -> int:
    """Loads of a lane for a row: 8 values of z and 8 of dy, 4 of dy with a gate, up to 16 bytes each."""
    return (3 if gated else 4) if fp32 else 2


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sums", [False, True])
def test_first_row_waits_for_its_own_loads(kernels, sums, gated, fp32):  # noqa: F811
    name = f"15act_grad_kernelI{'f' if fp32 else 'DF16b'}Lb{int(sums)}ELb{int(gated)}ELb1EE"
    (body,) = [b for k, b in kernels.items() if name in k]
    each = row_loads(gated, fp32)
    loads = [i for i, ins in enumerate(body) if ins.startswith("global_load") and ins.endswith(" nt")]
    assert len(loads) == ROWS * each
    waits = [re.search(r"vmcnt\((\d+)\)", ins) for ins in body[loads[-1]:] if ins.startswith("s_waitcnt")]
    first = [int(w.group(1)) for w in waits if w][:2]  # (dy, then z of the first row)
    assert min(first) >= (ROWS - 1) * each, first
