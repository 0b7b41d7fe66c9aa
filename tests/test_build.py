"""The build's guard of the kernels that move registers between warps with
setmaxnreg: a kernel launched with too few registers must never be linked."""
import os
import stat

import pytest

from block_sparse_approximate_b200 import build as bld


def _log(kernel, regs, arguments="ILi128EEEvi"):
    name = f"_ZN2sa12_GLOBAL__N_1{len(kernel)}{kernel}{arguments}"
    return (f"ptxas info    : Compiling entry function '{name}' for 'sm_100a'\n"
            f"ptxas info    : Function properties for {name}\n"
            "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
            f"ptxas info    : Used {regs} registers, used 2 barriers\n")


PAGED, ATTN, LINMIX = "paged_attn_tc_kernel", "attn_tc_kernel", "attn_tc_linmix_kernel"


def test_register_check_names_the_kernel():
    bld._check_tc_registers("paged_attn_tc.cu", _log(PAGED, 168) + _log(PAGED, 255, "ILi64EEEvi"))
    bld._check_tc_registers("attn_tc.cu", _log("block_pool_kernel", 20) + _log(ATTN, 158) + _log(LINMIX, 168))
    for src, log, name in (("paged_attn_tc.cu", _log(PAGED, 168) + _log(PAGED, 167, "ILi64EEEvi"), PAGED),
                           ("attn_tc.cu", _log(ATTN, 157) + _log(LINMIX, 168), ATTN),
                           ("attn_tc.cu", _log(ATTN, 168) + _log(LINMIX, 100), LINMIX)):
        with pytest.raises(RuntimeError, match=rf"\b{name} launches with \d+ registers"):
            bld._check_tc_registers(src, log)


@pytest.mark.parametrize("log", ["", _log(PAGED, 168).replace("Used 168 registers", "no figure"),
                                 _log("paged_combine_kernel", 168), _log(ATTN, 168)],
                         ids=["empty", "no_count", "another_kernel", "shorter_name"])
def test_register_check_needs_its_kernel(log):
    # a log that says nothing of the kernel is no proof
    with pytest.raises(RuntimeError, match=PAGED):
        bld._check_tc_registers("paged_attn_tc.cu", log)
    with pytest.raises(RuntimeError, match=LINMIX):
        bld._check_tc_registers("attn_tc.cu", _log(ATTN, 168))


@pytest.fixture
def small_tree(tmp_path, monkeypatch):
    """A tree of one guarded source, with a compiler that reports the register count in the file `regs`."""
    (tmp_path / "regs").write_text("168")
    src = tmp_path / "paged_attn_tc.cu"
    src.write_text("// source")
    log = _log(PAGED, "REGS")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text("#!/bin/bash\n"
                    'for a in "$@"; do [ "$last" = -o ] && out=$a; last=$a; done\n'
                    f'echo object > "$out"\ncat <<E | sed s/REGS/$(cat {tmp_path}/regs)/ >&2\n{log}E\n')
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(bld, "NVCC", str(nvcc))
    monkeypatch.setattr(bld, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(bld, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(bld, "_sources", lambda: [str(src)])
    monkeypatch.setattr(bld, "_headers", lambda: [])
    return tmp_path


def test_a_kernel_that_fails_the_check_is_not_linked_by_building_again(small_tree):
    (small_tree / "regs").write_text("160")
    for _ in range(2):
        with pytest.raises(RuntimeError, match="160 registers"):
            bld.build()
        assert not os.path.exists(bld.LIB) and not os.listdir(bld.BUILD)
    (small_tree / "regs").write_text("168")
    assert os.path.exists(bld.build())
    # a later source that fails leaves the object that passed; it stays older than the source
    os.utime(small_tree / "paged_attn_tc.cu", (4e9, 4e9))
    (small_tree / "regs").write_text("160")
    for _ in range(2):
        with pytest.raises(RuntimeError, match="160 registers"):
            bld.build()
    assert os.listdir(bld.BUILD) == ["paged_attn_tc.o"]


def test_bench_traffic_figure_describes_the_present_kernel():
    # the DRAM bytes of the attention kernel were captured on the sources as they are (bench.py reports null otherwise)
    import bench
    assert bench.attn_traffic_bytes() is not None
