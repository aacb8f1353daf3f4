"""The order of copies and stores in the assembly of the MXFP4 product with
several tiles a block (built here from source, no GPU needed).

Such a block issues the next tile's first copies into LDS in front of a tile's
stores and later waits with s_waitcnt vmcnt(16): all but the last 16 accesses
are done then, which covers the copies only if at least 16 stores of the wave
lie behind every one of them."""

import os
import re

import pytest

from tests.test_isa_cpu import CSRC, _device_asm

STORES = 16  # of a wave and tile: 4 groups of 32 rows, 8 rows an instruction


@pytest.fixture(scope="module")
def kernels():
    asm = _device_asm(os.path.join(CSRC, "linear.hip"))
    found = {}
    for m in re.finditer(r"^(_ZN\S*linear_gemm_kernelILb([01])ELi256ELi256\S*Lb1EE\S*):.*?^\.Lfunc_end", asm, re.S | re.M):
        found["mxfp4" if m.group(2) == "1" else "bf16"] = [
            line.split(";", 1)[0].strip() for line in m.group(0).splitlines()]
    assert sorted(found) == ["bf16", "mxfp4"]
    return found


@pytest.mark.parametrize("rows", ["bf16", "mxfp4"])
def test_stores_stay_behind_the_next_tiles_copies(kernels, rows):
    code = kernels[rows]
    copies = [i for i, c in enumerate(code) if c.startswith("buffer_load") and c.endswith("lds")]
    stores = [i for i, c in enumerate(code) if re.match(r"(global|flat|buffer)_store", c)]
    waits = [i for i, c in enumerate(code) if re.fullmatch(rf"s_waitcnt vmcnt\({STORES}\)", c)]
    assert copies and stores and waits
    # the copies of the loop and of the next tile come first, then the stores of a tile
    assert max(copies) < min(stores) and max(waits) < max(copies)
    # of whole rows one 16-byte store (bf16) or two (float32) for every eight rows
    wide = [i for i in stores if code[i].split()[0].endswith("_dwordx4")]
    assert len(wide) == 3 * STORES
