"""What the kernels' sources promise and no run can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "non_gated_relu_b200", "csrc")


def code(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_read_only_loads_of_what_a_launch_before_may_write():
    """The read-only path (__ldg, ld.global.nc, const with __restrict__ in a kernel's
    arguments) wants memory that nobody writes while the grid lives.  With programmatic
    launches a grid may be resident while the one before it still writes codes, scales,
    logits, rows and ids."""
    for name in ("gate.cuh", "gemm_f8.cuh", "gemm_f8s.cuh", "gemv_f8.cuh", "quant_f8.cuh"):
        text = code(name)
        assert "__ldg" not in text and ".nc" not in text, name
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", text), name
    # the gather's x is the caller's, or was complete three launches before
    text = code("permute.cuh")
    assert "__ldg" not in text and ".nc" not in text
    kernels = re.findall(r"__global__.*?\{", text, flags=re.S)
    assert len(kernels) == 5
    for k in kernels:
        for arg in re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", k):
            assert "permute_gather" in k and arg == "x", (arg, k)
    cast = re.findall(r"__global__ void cast_output\w*\((.*?)\)", code("nh_moe.cu"), flags=re.S)
    assert len(cast) == 2 and not any("__restrict__" in c for c in cast)


def test_only_fp8_products_need_the_fp8_kernels():
    """A build or device that the FP8 products do not fit refuses those calls alone: the
    setup that every other call waits for does not look at their kernels."""
    text = code("nh_moe.cu")
    body = text[text.index("static nh_status set_attrs("):text.index("static nh_status set_f8_attrs(")]
    assert "f8" not in body.lower()
    assert len(re.findall(r"\bf8_device_setup\(&dev\)", text)) == 0
    api = code("api_f8.cuh")
    entry = {m.group(1): m.group(0) for m in re.finditer(
        r"^(?:static )?nh_status (\w+)\([^{]*\{.*?^\}", api, flags=re.S | re.M)}
    for name in ("nh_fp8_linear", "f8_experts", "f8_shared"):
        assert "f8_device_setup(&dev)" in entry[name], name
    for name in ("nh_fp8_quantize", "nh_fp8_quantize_weight"):
        assert "f8_device_setup" not in entry[name], name
