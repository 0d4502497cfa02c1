"""The kernels that the products with microscaled weights launch, on the host:
the forms that the GPU tests are written for, and what goes before them."""
import mx_choice as C


def test_gpu_tests_take_the_kernels_they_name(tmp_path):
    import test_gpu_mx_kernels as G
    cases = G.calls()
    got = C.launches(tmp_path, [call for _, call in cases])
    assert len(got) == len(cases)
    off = [(name, call, launched) for (name, call), launched in zip(cases, got) if launched[-1] != name]
    assert not off, off[:5]
    # every mode of every form has a case
    names = {name for name, _ in cases}
    assert {f"{form}_{mode}" for form in ("large", "medium") for mode in ("dense", "adapted", "grouped", "gated")} <= names
    assert {"few_dense16", "few_dense32", "few_dense64", "few_adapted16", "few_adapted32", "few_adapted64", "few_grouped16", "few_gated16",
            "generic", "generic_gated"} <= names
