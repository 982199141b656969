"""Tile shapes that the ragged kernel's loads cannot serve are refused when it is compiled."""
import os
import subprocess

import pytest

from moe_w4a16_grouped_amd import build

SOURCE = """#include "ragged_gemm.h"
namespace moe {{
hipError_t launch(const RaggedArgs& a, hipStream_t s) {{ return launch_ragged_cfg<ElemF16, {mode}, MOE_EPI_NONE, {shape}>(a, s); }}
}}
"""


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("mode,shape,message", [
    ("kFwd", "TileShape<16, 64, 1, 2, 128, 2>", None),
    # 6 loads of a step's rows by 4 waves: two waves have a second one
    ("kDx", "TileShape<48, 128, 1, 4, 128, 2>", "every wave has all its loads"),
    ("kFwd", "TileShape<64, 192, 1, 4, 64, 2>", None),
    ("kFwd", "TileShape<64, 160, 1, 4, 64, 2>", "every wave has all its loads"),
])
def test_shapes(tmp_path, mode, shape, message):
    src = tmp_path / "shape.hip"
    src.write_text(SOURCE.format(mode=mode, shape=shape))
    run = subprocess.run([build.HIPCC, *build.FLAGS, "-O0", "-fsyntax-only", str(src)], capture_output=True, text=True, timeout=300)
    if message is None:
        assert run.returncode == 0, run.stderr
    else:
        assert run.returncode != 0 and message in run.stderr, run.stderr
