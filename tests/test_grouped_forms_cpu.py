"""The cases of test_gpu_grouped_forms run the instance that they are meant for, and between them all that there are."""
import grouped_plan as plan
import test_gpu_grouped_forms as forms


def test_the_products_instances():
    assert [plan.forward(True, *c[:3]) for c in forms.FORWARD] == [c[-1] for c in forms.FORWARD]
    assert {c[-1] for c in forms.FORWARD} == {(8, 128), (8, 0), (4, 64), (4, 0), "few"}


def test_the_dense_products_instances():
    assert [plan.forward(False, 1, *c[:2]) for c in forms.DENSE] == [c[-1] for c in forms.DENSE]


def test_the_rows_gradients_instances():
    assert [plan.turned(E, P, K) for E, P, _, K, _ in forms.TURNED] == [c[-1] for c in forms.TURNED]
    assert {c[-1] for c in forms.TURNED} == {(8, 128), (4, 64), (4, 0)}


def test_the_weights_gradients_instances():
    assert [plan.dw_large(E, N, K) for E, _, N, K, _ in forms.WEIGHTS] == [c[-1] for c in forms.WEIGHTS]
    assert {c[-1] for c in forms.WEIGHTS} == {True, False}
