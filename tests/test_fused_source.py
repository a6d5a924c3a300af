"""CPU checks of what the sources of the fused kernels must keep to and no run can show."""
import os
import re

import pytest

import nvfp4_block_scaled_08_b200 as nv

CSRC = os.path.join(os.path.dirname(nv.__file__), "csrc")


def code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["norm.cu", "gemm_kernel.cuh", "gemm_epilogue.cuh"])
def test_no_constant_data_loads(name):
    """These kernels may start while the kernel before them still writes, so nothing is loaded as data that is
    constant while they run: such a load need not stay behind the wait for that kernel."""
    text = code(name)
    assert not re.findall(r"__ldg\b|\.nc\b|__constant__", text)
    # global loads without volatile are ordered by their address alone: only in load_weights, of pointers
    # that behind_wait() gave
    loose = re.findall(r"asm\s*\(\s*\"ld\.global[^;]*;", text)
    if name != "norm.cu":
        assert not loose
        return
    body = text[text.index("void load_weights"):]
    body = body[:body.index("\n}\n")]
    assert len(loose) == body.count("ld.global") == 3
    tied = set(re.findall(r"(\w+) = behind_wait\(a\.\w+\)", text))
    assert tied == {"w_n", "b_n", "w_post", "w_gate"}
    used = set(re.findall(r"load_weights\((\w+) \+ 8", text)) | set(re.findall(r"multiply<TPR, V>\(z, in, t, (\w+),", text))
    assert used == tied | {"weights"}                # `weights`: multiply's own parameter
    assert text.index("grid_dependency_wait();") < text.index("behind_wait(a.")


def test_a_timed_out_side_box_ends_the_tile_loop():
    """The epilogue's result decides about the next tile: after a time-out its boxes would be sent into buffers,
    and armed on barriers, that one is still on its way to."""
    text = code("gemm_kernel.cuh")
    call = text.index("ok = epi.finish(")
    end = text.index("});", call)
    assert re.match(r"\}\);\s*if \(!ok\) break;", text[end:]), text[end:end + 80]
    # and what is still pending is waited for behind the loop, before the shared memory is released
    assert text.index("epi.drain();") > end


def test_every_split_k_launch_drains_its_receive_barrier():
    """A CTA that has given up waits, bounded, for its peers' rows before its shared memory is released: with a
    receive region of its own and with the reused stage ring."""
    text = code("gemm_kernel.cuh")
    at = text.index("mbar_wait_drain(rx_bar, 0)")
    guards = re.findall(r"if constexpr \(([^;]*?)\) \{", text[:at])
    assert guards[-1] == "!Cfg::GROUPED && !Cfg::PAIR"
    assert text.rindex("if (warp == 4 && lane == 0 && args.splits > 1 && args.cluster_size > 1)", 0, at) > text.rindex(guards[-1], 0, at)


def test_quantisers_load_behind_the_wait():
    """The same of the quantisers that may start early: their input is loaded through behind_wait()."""
    core = code("quant_core.cuh")
    load = core[core.index("template <> struct InTraits<float>"):core.index("struct GlobalVecs")]
    assert "__ldg" not in load and load.count("ld_behind(p") == 3
    text = code("quantize.cu")
    for kernel in text.split("__global__")[1:]:
        if "grid_dependency_wait();" in kernel:
            body = kernel[kernel.index("grid_dependency_wait();"):]
            assert set(re.findall(r"GlobalVecs<T>(?: in)?\{([^,]*),", kernel)) == {"behind_wait(x)"}
            assert "behind_wait(x)" in body and "gs_other[" not in body and "__ldg" not in body
    assert "behind_wait(static_cast<const T*>(a.act))" in code("gemm_kernel.cuh")
