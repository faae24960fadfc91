"""The rows that the gated scan's kernels are given lie as the kernels read
them, whatever strides a caller leaves where they mean nothing: the library's
own host code, without a GPU."""
import glob
import os
import subprocess

from state_space_model_fwd_gb300 import _build

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "gated_rows_host.cu")


def test_rows_read_in_pairs_lie_on_pairs_boundaries(tmp_path):
    _build.build()
    if not glob.glob(os.path.join(_build.OBJ_DIR, "*.o")):  # only the library was kept
        _build.build(force=True)
    exe = str(tmp_path / "gated_rows_host")
    objects = sorted(glob.glob(os.path.join(_build.OBJ_DIR, "*.o")))
    flags = [f for f in _build.NVCC_FLAGS if f not in ("-O3", "-lineinfo")]
    subprocess.run([_build._nvcc(), *_build.ARCH, *flags, "-o", exe, SOURCE, *objects, "-cudart", "static"], check=True,
                   capture_output=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[:2000]
